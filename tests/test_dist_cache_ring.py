"""The ring inside a group with 8-bit K and V on gloo ranks on the CPU: real exchanges, the
kernel launches replaced by the fp64 oracle (as in test_dist_schedules.py, whose 16-bit ring
this one follows)."""
import numpy as np
import pytest
import torch
import torch.multiprocessing as mp

import oracle as O
from test_dist_schedules import HostOps, _free_port, _f64, _init, _run_ranks

E4M3 = torch.float8_e4m3fn


class HostCacheOps(HostOps):
    """The cache calls on the host: codes as bytes, so that what travels is what is attended."""

    def store(self, k, v, cache, stream=None):
        kc, vc, ks, vs = cache
        for x, codes, scale in ((k, kc, ks), (v, vc, vs)):
            for h in range(x.shape[1]):
                c, s = O.cache_store(_f64(x)[0, h], 0, np.zeros(tuple(x.shape[2:])), np.zeros(scale.shape[2]))
                codes[0, h] = torch.from_numpy(c).float().to(E4M3).view(torch.uint8)
                scale[0, h] = torch.from_numpy(s)

    def cache_workspace(self, q, cache):
        return None

    def attend_cache(self, q, cache, o, lse, workspace, stream=None):
        self.launches.append(None)
        k, v = (O.cache_values(_f64(c.view(E4M3).float()), _f64(s)) for c, s in (cache[::2], cache[1::2]))
        ro, rl = O.cache_attn(_f64(q), k, v, [k.shape[2]], self.scale)
        o.copy_(torch.from_numpy(ro))
        lse.copy_(torch.from_numpy(rl))


def _rank(rank, ws, port, cfg, out):
    dist = _init(rank, ws, port)
    try:
        from sequence_partition_attn_b200.dist import GroupRing, HostStagedExchange
        N_blk, H, D = cfg
        g = torch.Generator().manual_seed(9)
        full = [torch.randn(1, H, N_blk * ws, D, generator=g) for _ in range(3)]
        ops = HostCacheOps(1.0 / np.sqrt(D))
        ring = GroupRing(ops, HostStagedExchange(), None, N_blk, H, D, 1, dtype=torch.float32,
                         device="cpu", kv_bits=8)
        for w in ring.wire:
            w[0].fill_(0x7F)               # a block read before it arrives shows as NaN
        blk = [x[:, :, rank * N_blk:(rank + 1) * N_blk].contiguous() for x in full]
        first = [t.clone() for t in ring.run(*blk)]
        o, lse = ring.run(*blk)            # buffers are reused
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
        out.put((rank, o.numpy().copy(), lse.numpy().copy(), ring.lse_part.numpy().copy(), len(ops.launches)))
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("ws,cfg", [(1, (10, 1, 8)), (2, (70, 2, 16)), (3, (64, 1, 8)), (4, (130, 2, 8))])
def test_eight_bit_ring_on_gloo_ranks(ws, cfg):
    N_blk, H, D = cfg
    res = _run_ranks(_rank, ws, _free_port(), cfg, mp.get_context("spawn").Queue())
    g = torch.Generator().manual_seed(9)
    q, k, v = (_f64(torch.randn(1, H, N_blk * ws, D, generator=g)) for _ in range(3))
    # every block goes through the cache on its own rank
    held = []
    for x in (k, v):
        y = np.empty_like(x)
        for s in range(ws):
            for h in range(H):
                rows = x[0, h, s * N_blk:(s + 1) * N_blk]
                c, sc = O.cache_store(rows, 0, np.zeros_like(rows), np.zeros(-(-N_blk // 64)))
                y[0, h, s * N_blk:(s + 1) * N_blk] = O.cache_values(c, sc)
        held.append(y)
    ro, rl = O.cache_attn(q, *held, [N_blk * ws], 1.0 / np.sqrt(D))
    for rank, o, lse, lse_part, launches in res:
        rows = slice(rank * N_blk, (rank + 1) * N_blk)
        # states and results are fp32: 2^-24 of values and logarithms below 16
        assert np.abs(o - ro[:, :, rows]).max() <= 1e-5 and np.abs(lse - rl[:, :, rows]).max() <= 1e-5
        assert launches == 2 * ws and lse_part.shape[0] == ws
        for s in range(ws):
            blk = [x[:, :, s * N_blk:(s + 1) * N_blk] for x in held]
            want = O.cache_attn(q[:, :, rows], *blk, [N_blk], 1.0 / np.sqrt(D))[1]
            assert np.abs(lse_part[s] - want).max() <= 1e-5


def test_block_bytes_hold_codes_and_scales_apart():
    from sequence_partition_attn_b200.dist import cache_bytes, cache_views
    for H, N, D in [(1, 1, 64), (3, 65, 128), (2, 9450, 128)]:
        buf = torch.zeros(cache_bytes(H, N, D), dtype=torch.uint8)
        views = cache_views(buf, H, N, D)
        assert [tuple(x.shape) for x in views[:2]] == [(1, H, N, D)] * 2
        assert [tuple(x.shape) for x in views[2:]] == [(1, H, -(-N // 64))] * 2
        assert sum(x.numel() * x.element_size() for x in views) == buf.numel()
        at = [x.data_ptr() - buf.data_ptr() for x in views]
        assert at[:2] == [0, H * N * D] and at[1] % 16 == 0 and at[2] % 16 == 0 and at == sorted(at)
        for i, x in enumerate(views):
            x.fill_(i + 1)
        assert all(bool((x == i + 1).all()) for i, x in enumerate(views))


def test_refusals():
    import datetime
    import os
    import torch.distributed as dist
    from sequence_partition_attn_b200.dist import GroupRing
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(_free_port()))
    dist.init_process_group("gloo", rank=0, world_size=1, timeout=datetime.timedelta(seconds=30))
    try:
        with pytest.raises(ValueError):
            GroupRing(None, None, None, 64, 2, 64, 2, device="cpu", kv_bits=8)
        with pytest.raises(ValueError):
            GroupRing(None, None, None, 64, 2, 64, 1, device="cpu", kv_bits=4)
    finally:
        dist.destroy_process_group()
