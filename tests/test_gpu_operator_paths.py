"""The framework's own paths through the backward pass and the 8-bit cache, and the sizes that
reach the kernels' other forms: many partitions, many requests, long caches."""
import datetime
import os

import numpy as np
import pytest
import torch
import torch.multiprocessing as mp

import bounds
import oracle as O
import sequence_partition_attn_b200 as pa
from test_gpu_backward import compare as compare_grads
from test_gpu_backward import even, f64, grads, make
from test_gpu_cache import attend, compare, empty_cache, make_cache, queries, starts
from test_gpu_dist import _free_port, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = pa.Context(0)
    yield c
    c.close()


# ------------------------------------------------------------------ the step's backward
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_backward_follows_its_forward(ctx, dtype):
    """run() with cached states, then backward(): the gradients of the fresh pairs' share of the
    merged state."""
    from sequence_partition_attn_b200.step import AttentionStep
    B, H, N, D, G = 1, 2, 500, 64, 1
    off = even(N, 5)
    fresh = np.eye(5, dtype=np.uint8)
    fresh[1, 3] = fresh[4, 0] = 1
    t = make(B, H, N, D, dtype, off, G, fresh, 21, dlse=True)
    step = AttentionStep(ctx, B, H, N, D, off, G, fresh, dtype=t["q"].dtype)
    g = torch.Generator().manual_seed(22)
    for n in ("q", "k", "v"):
        getattr(step, n).copy_(t[n])
    k_prev, v_prev = (torch.randn(B, H, N, D, generator=g).to(t["q"]) for _ in range(2))
    step.fill_cache(k_prev, v_prev)
    step.run()
    out = [torch.full_like(t["q"], float("nan")) for _ in range(3)]
    step.backward(t["do"], *out, dlse=t["dlse"])
    ctx.sync_status()
    t["o"], t["lse"] = step.o, step.lse
    compare_grads(t, out, step.delta, off, G, fresh, dtype)
    again = [torch.empty_like(x) for x in out]
    step.backward(t["do"], *again, dlse=t["dlse"], q=t["q"], k=t["k"], v=t["v"], o=step.o, lse=step.lse)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


# ------------------------------------------------------------------ many partitions
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P,G", [(32, 1), (33, 1), (128, 1), (128, 5)])
def test_many_partitions(ctx, dtype, P, G):
    N, D = 700, 64
    off = np.sort(np.concatenate([[0, N], np.random.default_rng(P).integers(0, N + 1, P - 1)]))
    QG = -(-P // G)
    fresh = (np.random.default_rng(G).random((QG, QG)) < 0.3).astype(np.uint8)
    t = make(1, 2, N, D, dtype, off, G, fresh, 30 + P)
    out, delta = grads(ctx, t, off, G, fresh)
    ctx.sync_status()
    compare_grads(t, out, delta, off, G, fresh, dtype)


# ------------------------------------------------------------------ many requests and rows
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [300, 700])                  # whole units, and shares of them
@pytest.mark.parametrize("B,H,Hk,Nq", [(70, 2, 2, 1), (33, 6, 2, 3), (2, 2, 1, 150), (3, 1, 1, 33), (40, 24, 24, 1)])
def test_many_requests_and_rows(ctx, dtype, B, H, Hk, Nq, M):
    D = 64
    lens = [int(x) for x in np.random.default_rng(B).integers(0, M + 1, B)]
    lens[0], lens[-1] = 0, M
    cache = make_cache(ctx, B, Hk, M, D, 40 + B)
    q = queries(B, H, Nq, D, dtype, 41)
    o, lse = attend(ctx, q, cache, starts(lens))
    ctx.sync_status()
    compare(q, cache, lens, o, lse, dtype)


@pytest.mark.parametrize("Nq", [1, 20, 40])
def test_cache_offsets_past_32_bits(ctx, Nq):
    """A second request whose codes lie past 2^31 bytes: zeros but for its last block, whose
    scores outweigh the rest.  lse and o of the held tokens follow in closed form."""
    D, M, T = 128, 9_000_020, 64
    kc, vc = (torch.zeros(2, 1, M, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(2, 1, -(-M // 64), device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(50)
    q = torch.randn(2, 1, Nq, D, generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn(2, 1, T, D, generator=g).mul(s).to(torch.bfloat16).cuda() for s in (6.0, 1.0))
    pa.pa_cache_store(ctx, k, v, starts([0, M - T]), kc, vc, ks, vs)
    o, lse = attend(ctx, q, (kc, vc, ks, vs), starts([T, M]))
    ctx.sync_status()
    tail = (M - T) % 64                                    # the rows straddle two cache blocks
    kk, vv = ([x[0, :, :T], x[1, :, M - T:]] for x in (kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)))
    for b, base in ((0, 0), (1, (M - T) // 64)):
        sc = [np.repeat(f64(s[b, 0, base:base + 2]), 64)[(tail if b else 0):][:T] for s in (ks, vs)]
        kf, vf = (f64(x[b].float())[0] * s[:, None] for x, s in zip((kk, vv), sc))
        for x, y in ((kf, k), (vf, v)):                     # e4m3: 2^-4, or half its smallest step
            assert (np.abs(x - f64(y)[b, 0]) <= 2.0 ** -4 * np.abs(f64(y)[b, 0]) + 2.0 ** -10 * max(sc[0].max(), sc[1].max())).all()
        qf = f64(q)[b, 0]
        s = D ** -0.5 * qf @ kf.T
        m = np.maximum(s.max(1, keepdims=True), 0.0)
        rest = (M - T if b else 0) * np.exp(-m[:, 0])
        z = np.exp(s - m).sum(1) + rest
        want_l = m[:, 0] + np.log(z)
        want_o = (np.exp(s - m) / z[:, None]) @ vf
        mag = (np.exp(s - m) / z[:, None]) @ np.abs(vf)
        # scores: 2 D u sum|q k|; M equal terms summed in 128-term groups, 2 (n + 4) u with n the
        # longest chain of one accumulator (fewer than M / 128 groups)
        chain = 2 * (M / 128 + 132) * bounds.U if b else 2 * 132 * bounds.U
        es = (2 * D * bounds.U * D ** -0.5 * np.abs(qf) @ np.abs(kf).T).max(1) + 8 * bounds.U * np.abs(s).max(1) + 2.0 ** -21
        # the zero tokens' weight is 1/z each: its rounding counts as theirs do
        rel = 2 * es + 2 * chain
        assert (np.abs(f64(lse)[b, 0] - want_l) <= rel + 4 * bounds.U * np.abs(want_l) + 2.0 ** -21).all()
        tol = (rel + bounds.BF16)[:, None] * mag + bounds.BF16 * (np.abs(want_o) + mag * 2.0 ** -6) + 1e-30
        assert (np.abs(f64(o)[b, 0] - want_o) <= tol).all()


# ------------------------------------------------------------------ the ring in 8 bits
def _ring_rank(rank, ws, port, cfg, out):
    import torch.distributed as dist
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=ws, timeout=datetime.timedelta(seconds=120))
    try:
        from sequence_partition_attn_b200.dist import DeviceOps, GroupRing, HostStagedExchange
        torch.cuda.set_device(0)
        c = pa.Context(0)
        N_blk, H, D = cfg
        ring = GroupRing(DeviceOps(c), HostStagedExchange(), None, N_blk, H, D, 1, device="cuda:0", kv_bits=8)
        for w in ring.wire:
            w[0].fill_(0x7F)
        full = _inputs(4, (1, H, N_blk * ws, D))
        blk = [x[:, :, rank * N_blk:(rank + 1) * N_blk].contiguous().cuda() for x in full]
        o, lse = ring.run(*blk)
        c.sync_status()
        out.put((rank, o.float().cpu().numpy(), lse.cpu().numpy()))
        c.close()
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("cfg", [(640, 2, 128), (77, 3, 64), (20, 1, 64)])
def test_eight_bit_ring_two_ranks_on_one_gpu(cfg):
    N_blk, H, D = cfg
    ws, scale = 2, D ** -0.5
    queue = mp.get_context("spawn").Queue()
    pc = mp.start_processes(_ring_rank, args=(ws, _free_port(), cfg, queue), nprocs=ws, join=False, start_method="spawn")
    res = [queue.get(timeout=600) for _ in range(ws)]
    while not pc.join(timeout=60):
        pass
    q, k, v = (x.double().numpy() for x in _inputs(4, (1, H, N_blk * ws, D)))
    held = []
    for x in (k, v):
        y = np.empty((ws, 1, H, N_blk, D))
        for s in range(ws):
            for h in range(H):
                rows = x[0, h, s * N_blk:(s + 1) * N_blk]
                c, sc = O.cache_store(rows, 0, np.zeros_like(rows), np.zeros(-(-N_blk // 64)))
                y[s, 0, h] = O.cache_values(c, sc)
        held.append(y)
    for rank, o, lse in res:
        qr = q[:, :, rank * N_blk:(rank + 1) * N_blk]
        part = [O.cache_attn(qr, held[0][s], held[1][s], [N_blk], scale) for s in range(ws)]
        tol = [bounds.attention(qr, held[0][s], held[1][s], [N_blk], scale, bounds.BF16) for s in range(ws)]
        ls = np.stack([p[1] for p in part])
        top = ls.max(0)
        z = np.exp(ls - top).sum(0)
        w = np.exp(ls - top) / z
        want_l = top + np.log(z)
        want_o = sum(w[s][..., None] * part[s][0] for s in range(ws))
        el = np.stack([t[1] for t in tol]).max(0)
        bounds.check("lse", lse, want_l, el + 8 * bounds.U * (np.abs(want_l) + 1) + 2.0 ** -21)
        # weights err by what the states' lse do, twice (own and sum), plus the merge's exponentials
        ew = 2 * el + 2.0 ** -20
        e = sum(w[s][..., None] * (tol[s][0] + ew[..., None] * (np.abs(part[s][0]) + tol[s][0])) for s in range(ws))
        bounds.check("o", o, want_o, e + bounds.BF16 * (np.abs(want_o) + e) + 2.0 ** -126)
