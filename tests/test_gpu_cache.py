"""The 8-bit K/V cache: stored codes and scales equal the oracle's, and attention over the
cache is within the bounds of the roundings made (tests/bounds.py)."""
import numpy as np
import pytest
import torch

import bounds
import oracle as O
import sequence_partition_attn_b200 as pa

pytestmark = pytest.mark.gpu
DT = {"f32": (torch.float32, bounds.F32), "bf16": (torch.bfloat16, bounds.BF16)}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ctx():
    c = pa.Context(0)
    yield c
    c.close()


def f64(t):
    return t.detach().double().cpu().numpy() if t.dtype != E4M3 else t.float().double().cpu().numpy()


def empty_cache(B, Hk, M, D):
    """Codes and scales full of NaN: a cache needs no initialisation."""
    nb = -(-M // pa.PA_CACHE_BLOCK)
    codes = [torch.full((B, Hk, M, D), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    return codes + [torch.full((B, Hk, nb), float("nan"), device="cuda") for _ in range(2)]


def starts(s):
    return torch.tensor(s, dtype=torch.int32, device="cuda")


def same(a, b):
    return np.array_equal(a, b, equal_nan=True)


# ------------------------------------------------------------------ store
STORES = [  # B, Hk, T, M, D, start, dtype
    (1, 1, 1, 1, 64, [0], "bf16"), (1, 2, 64, 64, 128, [0], "f32"), (2, 1, 65, 130, 64, [0, 65], "bf16"),
    (3, 2, 1, 200, 128, [0, 63, 199], "bf16"), (2, 3, 1, 100, 64, [64, 99], "f32"),
    (2, 2, 130, 400, 128, [7, 270], "bf16"), (1, 1, 63, 127, 128, [64], "f32"), (1, 5, 700, 777, 64, [77], "bf16"),
]


@pytest.mark.parametrize("case", range(len(STORES)))
def test_store_equals_the_oracle(ctx, case):
    """Behind earlier tokens of a smaller and of a larger spread, so that scales grow and stay."""
    B, Hk, T, M, D, st, dtype = STORES[case]
    g = torch.Generator().manual_seed(case)
    cache = empty_cache(B, Hk, M, D)
    kc, vc, ks, vs = cache
    held = [(torch.randn(B, Hk, M, D, generator=g) * s).cuda() for s in (0.01, 40.0)]
    pa.pa_cache_store(ctx, held[0], held[1], None, kc, vc, ks, vs)
    before = [f64(x) for x in cache]
    k, v = (torch.randn(B, Hk, T, D, generator=g).to(DT[dtype][0]).cuda() for _ in range(2))
    pa.pa_cache_store(ctx, k, v, starts(st), kc, vc, ks, vs)
    ctx.sync_status()
    for codes, scale, x, c0, s0 in ((kc, ks, k, before[0], before[2]), (vc, vs, v, before[1], before[3])):
        for b in range(B):
            for h in range(Hk):
                wc, ws = O.cache_store(f64(x)[b, h], st[b], c0[b, h], s0[b, h])
                assert same(f64(scale)[b, h], ws)
                assert same(f64(codes)[b, h], wc)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_first_store_and_untouched_rest(ctx, dtype):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(1, 2, 100, 64, generator=g).to(DT[dtype][0]).cuda()
    kc, vc, ks, vs = empty_cache(1, 2, 300, 64)
    pa.pa_cache_store(ctx, x, x, None, kc, vc, ks, vs)
    ctx.sync_status()
    for h in range(2):
        wc, ws = O.cache_store(f64(x)[0, h], 0, np.full((300, 64), np.nan), np.full(5, np.nan))
        assert same(f64(kc)[0, h], wc) and same(f64(ks)[0, h], ws)
    assert torch.equal(kc.view(torch.uint8), vc.view(torch.uint8))
    assert bool((kc.view(torch.uint8)[:, :, 100:] == 0x7F).all()) and bool(ks[:, :, 2:].isnan().all())


def test_tokens_one_at_a_time_keep_the_bound(ctx):
    """Re-rounding under a growing scale: each code is off by at most half an e4m3 step of its
    first rounding plus one of each growth, and the final scale is that of storing all at once."""
    g = torch.Generator().manual_seed(3)
    M, D = 70, 128
    x = (torch.randn(1, 1, M, D, generator=g) * torch.logspace(-3, 1, M)[:, None]).to(torch.bfloat16).cuda()
    cache, once = empty_cache(1, 1, M, D), empty_cache(1, 1, M, D)
    codes, scale = np.full((M, D), np.nan), np.full(2, np.nan)
    for t in range(M):
        row = x[:, :, t:t + 1].contiguous()
        pa.pa_cache_store(ctx, row, row, starts([t]), cache[0], cache[1], cache[2], cache[3])
        codes, scale = O.cache_store(f64(row)[0, 0], t, codes, scale)
    pa.pa_cache_store(ctx, x, x, None, *once)
    ctx.sync_status()
    assert same(f64(cache[0])[0, 0], codes) and same(f64(cache[2])[0, 0], scale)
    assert torch.equal(cache[2], once[2]) and torch.equal(cache[3], once[3])
    val = O.cache_values(codes, scale)
    # normal range: 2^-4 per rounding, and normal codes do not change when the scale grows by a
    # power of two; below it half the smallest step, 2^-10 of the final scale, per growth (< 16)
    assert (np.abs(val - f64(x)[0, 0]) <= 2.0 ** -4 * np.abs(f64(x)[0, 0]) + 16 * 2.0 ** -10 * scale[np.arange(M) // 64][:, None]).all()


def test_extreme_values(ctx):
    D = 64
    rows = torch.zeros(1, 1, 64 * 8, D)
    big = 3.0e38
    rows[0, 0, 0, 3] = big                                       # the largest scales
    rows[0, 0, 64, :4] = torch.tensor([448.0, -448.0, 1.0, 0.0])
    rows[0, 0, 128, :2] = torch.tensor([448.0001, 7.0])          # just above: the next power
    rows[0, 0, 192, 0] = 1e-42                                   # below 2^-126 * 448: the smallest scale
    rows[0, 0, 256, :3] = torch.tensor([float("inf"), 2.0, float("-inf")])
    rows[0, 0, 320, :2] = torch.tensor([float("nan"), 2.0])
    rows[0, 0, 448, 0] = -0.0                                    # and a block of zeros
    x = rows.cuda()
    kc, vc, ks, vs = empty_cache(1, 1, 512, D)
    pa.pa_cache_store(ctx, x, x, None, kc, vc, ks, vs)
    ctx.sync_status()
    wc, ws = O.cache_store(f64(x)[0, 0], 0, np.zeros((512, D)), np.zeros(8))
    assert same(f64(kc)[0, 0], wc) and same(f64(ks)[0, 0], ws)
    assert float(ks[0, 0, 1]) == 1.0 and float(ks[0, 0, 2]) == 2.0 and float(ks[0, 0, 3]) == 2.0 ** -126
    assert float(ks[0, 0, 6]) == 0.0 and float(ks[0, 0, 7]) == 0.0


def test_start_outside_the_cache_is_reported_and_writes_nothing(ctx):
    x = torch.ones(3, 1, 10, 64, dtype=torch.bfloat16, device="cuda")
    cache = empty_cache(3, 1, 100, 64)
    pa.pa_cache_store(ctx, x, x, starts([91, 90, -1]), *cache)
    with pytest.raises(pa.PAError) as e:
        ctx.sync_status()
    assert e.value.code == -1
    ctx.sync_status()                                            # reported once
    u = cache[0].view(torch.uint8)
    assert bool((u[0] == 0x7F).all()) and bool((u[2] == 0x7F).all())
    assert bool((u[1, :, 90:] == 0x78).all()) and float(cache[2][1, 0, 1]) == 2.0 ** -8     # 1 = 256 * 2^-8


# ------------------------------------------------------------------ attention
def make_cache(ctx, B, Hk, M, D, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(B, Hk, M, D, generator=g).mul(spread).cuda() for _ in range(2))
    cache = empty_cache(B, Hk, M, D)
    pa.pa_cache_store(ctx, k, v, None, *cache)
    return cache


def values(cache):
    return O.cache_values(f64(cache[0]), f64(cache[2])), O.cache_values(f64(cache[1]), f64(cache[3]))


def attend(ctx, q, cache, lens, **kw):
    o = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    if kw.get("stream") is not None:
        kw["stream"].wait_stream(torch.cuda.current_stream())    # which fills the outputs
    pa.pa_cache_attn(ctx, q, *cache, lens, o, lse, **kw)
    return o, lse


def queries(B, H, Nq, D, dtype, seed, gain=1.0):
    g = torch.Generator().manual_seed(1000 + seed)
    return torch.randn(B, H, Nq, D, generator=g).mul(gain).to(DT[dtype][0]).cuda()


def compare(q, cache, lens, o, lse, dtype, scale=None):
    scale = q.shape[3] ** -0.5 if scale is None else scale
    k, v = values(cache)
    B, M = k.shape[0], k.shape[2]
    n = [M] * B if lens is None else [min(max(x, 0), M) for x in lens]
    for b in range(B):
        k[b, :, n[b]:], v[b, :, n[b]:] = 0, 0                   # may be NaN there
    wo, wl = O.cache_attn(f64(q), k, v, n, scale)
    eo, el = bounds.attention(f64(q), k, v, n, scale, DT[dtype][1])
    bounds.check("lse", f64(lse), wl, el)
    bounds.check("o", f64(o), wo, eo)


ATTN = [  # B, H, Hk, Nq, M, D, lens
    (1, 1, 1, 1, 1, 64, None), (1, 1, 1, 1, 1, 128, None), (2, 2, 2, 1, 63, 64, [63, 1]),
    (3, 4, 1, 1, 64, 128, [0, 64, 33]), (2, 8, 2, 1, 65, 64, [65, 64]), (1, 5, 1, 3, 127, 128, None),
    (2, 3, 3, 1, 1000, 128, [1000, 999]), (1, 16, 2, 2, 129, 64, None), (1, 17, 1, 1, 300, 128, None),
    (2, 6, 2, 11, 513, 64, [500, 0]), (1, 2, 1, 40, 777, 128, [640]), (1, 1, 1, 127, 200, 64, None),
    (1, 1, 1, 128, 128, 128, None), (2, 1, 1, 129, 257, 64, [256, 1]), (1, 2, 2, 300, 450, 128, [449]),
    (2, 4, 2, 200, 130, 64, [130, 0]), (1, 1, 1, 1, 5000, 128, [4097]), (1, 8, 1, 8, 2500, 64, None),
    (4, 1, 1, 65, 640, 128, [640, 0, 1, 577]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention_against_the_formulas(ctx, case, dtype):
    B, H, Hk, Nq, M, D, lens = ATTN[case]
    cache = make_cache(ctx, B, Hk, M, D, case)
    q = queries(B, H, Nq, D, dtype, case, gain=2.0)
    o, lse = attend(ctx, q, cache, None if lens is None else starts(lens))
    ctx.sync_status()
    compare(q, cache, lens, o, lse, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Nq", [1, 20, 200])
def test_tokens_behind_the_length_may_hold_anything(ctx, dtype, Nq):
    """NaN codes and NaN and infinite scales behind the length, and inside its last block."""
    B, Hk, M, D = 2, 2, 400, 128
    lens = [70, 256]
    cache = make_cache(ctx, B, Hk, M, D, 5)
    q = queries(B, 4, Nq, D, dtype, 5)
    want = attend(ctx, q, cache, starts(lens))
    for b, n in enumerate(lens):
        for i in range(2):
            cache[i].view(torch.uint8)[b, :, n:] = 0x7F
            cache[2 + i][b, :, -(-n // 64):] = float("inf") if i else float("nan")
    got = attend(ctx, q, cache, starts(lens))
    ctx.sync_status()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Nq", [1, 150])
@pytest.mark.parametrize("gain,spread", [(1e-3, 1e-6), (8.0, 3.0), (1e-20, 1e15), (1e15, 1e-14)])
def test_flat_peaked_and_far_scales(ctx, dtype, Nq, gain, spread):
    cache = make_cache(ctx, 1, 1, 333, 64, 6, spread)
    q = queries(1, 2, Nq, 64, dtype, 6, gain)
    o, lse = attend(ctx, q, cache, None)
    compare(q, cache, None, o, lse, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Nq", [1, 140])
def test_blocks_of_very_different_scales(ctx, dtype, Nq):
    """V blocks 2^40 apart, the weight on the small one: nothing of it may be lost."""
    M, D = 192, 64
    g = torch.Generator().manual_seed(7)
    k, v = torch.zeros(1, 1, M, D), torch.randn(1, 1, M, D, generator=g)
    k[0, 0, 64:128, 0] = 24.0
    v[0, 0, :64] *= 2.0 ** -20
    v[0, 0, 64:128] *= 2.0 ** -40
    v[0, 0, 128:] = 0
    cache = empty_cache(1, 1, M, D)
    pa.pa_cache_store(ctx, k.cuda(), v.cuda(), None, *cache)
    q = torch.zeros(1, 1, Nq, D)
    q[..., 0] = 16.0
    q = q.to(DT[dtype][0]).cuda()
    o, lse = attend(ctx, q, cache, None)
    compare(q, cache, None, o, lse, dtype)


def test_result_does_not_depend_on_the_company(ctx):
    """A request alone and in a batch, and repeated: the same bits."""
    cache = make_cache(ctx, 3, 2, 900, 128, 8)
    q = queries(3, 4, 1, 128, "bf16", 8)
    lens = [900, 450, 1]
    a = attend(ctx, q, cache, starts(lens))
    b = attend(ctx, q, cache, starts(lens))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_workspace_streams_and_graph(ctx):
    B, Hk, M, D = 2, 2, 3000, 128
    cache = make_cache(ctx, B, Hk, M, D, 9)
    q = queries(B, 4, 1, D, "bf16", 9)
    lens = starts([3000, 1234])
    want = attend(ctx, q, cache, lens)
    ws = [pa.cache_attn_workspace(ctx, q, cache[0]) for _ in range(2)]
    assert ws[0].numel() > 0
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [attend(ctx, q, cache, lens, workspace=w, stream=s) for w, s in zip(ws, streams) for _ in range(3)]
    own = attend(ctx, q, cache, lens, stream=streams[0])
    torch.cuda.synchronize()
    for x in got + [own]:
        assert all(torch.equal(a, b) for a, b in zip(want, x))
    # two graphs with scratch of their own; lengths are read at replay
    outs = [[torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")] for _ in range(2)]
    graphs = []
    for w, out in zip(ws, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pa.pa_cache_attn(ctx, q, *cache, lens, *out, workspace=w)
        graphs.append(graph)
    lens.copy_(starts([17, 0]))
    for s, graph in zip(streams, graphs):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    want = attend(ctx, q, cache, lens)
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    ctx.sync_status()


def test_append_and_attend_token_by_token(ctx):
    """A prompt, then single tokens: store and attend, in one captured graph per step."""
    B, H, Hk, M, D, n0 = 2, 4, 2, 160, 64, 60
    g = torch.Generator().manual_seed(10)
    k, v = (torch.randn(B, Hk, M, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    cache = empty_cache(B, Hk, M, D)
    pa.pa_cache_store(ctx, k[:, :, :n0].contiguous(), v[:, :, :n0].contiguous(), None, *cache)
    kn, vn = (torch.empty(B, Hk, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = queries(B, H, 1, D, "bf16", 10)
    at, lens = starts([n0] * B), starts([n0 + 1] * B)
    o, lse = torch.empty_like(q), torch.empty(B, H, 1, device="cuda")
    ws = pa.cache_attn_workspace(ctx, q, cache[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pa.pa_cache_store(ctx, kn, vn, at, *cache)
        pa.pa_cache_attn(ctx, q, *cache, lens, o, lse, workspace=ws)
    for t in range(n0, n0 + 8):
        kn.copy_(k[:, :, t:t + 1])
        vn.copy_(v[:, :, t:t + 1])
        graph.replay()
        torch.cuda.synchronize()
        compare(q, cache, [t + 1] * B, o, lse, "bf16")
        at.add_(1)
        lens.add_(1)
    ctx.sync_status()


def test_cache_states_merge_with_fresh_states_and_the_fresh_pairs_train(ctx):
    """The set together: far tokens in the 8-bit cache, near ones fresh; the states merge, and
    the backward pass differentiates the fresh part with the joint log-sum-exp."""
    B, H, N, D, far = 1, 2, 200, 64, 300
    g = torch.Generator().manual_seed(11)
    q, k, v, do = (torch.randn(B, H, N, D, generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    cache = make_cache(ctx, B, H, far, D, 11)
    P, off = 2, np.array([0, 100, N])
    of = torch.zeros(P, B, H, N, D, dtype=torch.bfloat16, device="cuda")
    lf = torch.zeros(P, B, H, N, device="cuda")
    oc, lc = torch.zeros_like(of), torch.full_like(lf, float("-inf"))
    fresh = np.eye(2, dtype=np.uint8)
    pa.pa_partition_attn(ctx, q, k, v, off, 1, fresh, of, lf)
    pa.pa_cache_attn(ctx, q, *cache, None, oc[1], lc[1])          # the far state, in both groups' reused slot
    oc[0], lc[0] = oc[1], lc[1]
    o, lse = torch.empty_like(q), torch.empty(B, H, N, device="cuda")
    pa.pa_merge_states(ctx, off, 1, fresh, of, lf, oc, lc, o, lse)
    out = [torch.empty_like(q) for _ in range(3)]
    pa.pa_attn_backward(ctx, q, k, v, o, lse, do, off, 1, fresh, *out, torch.empty_like(lse))
    ctx.sync_status()
    kk, vv = values(cache)
    scale = D ** -0.5
    qf, kf, vf = f64(q), f64(k), f64(v)
    for r in (slice(0, 100), slice(100, 200)):
        s = scale * np.concatenate([qf[:, :, r] @ kf[:, :, r].swapaxes(2, 3), qf[:, :, r] @ kk.swapaxes(2, 3)], axis=3)
        m = s.max(-1, keepdims=True)
        z = np.exp(s - m).sum(-1, keepdims=True)
        want = (np.exp(s - m) / z) @ np.concatenate([vf[:, :, r], vv], axis=2)
        # three bf16 roundings of values up to max|v| (weights, states, output)
        assert np.abs(f64(o)[:, :, r] - want).max() <= 3 * 2.0 ** -8 * max(np.abs(vf).max(), np.abs(vv).max())
        assert np.abs(f64(lse)[:, :, r] - (m + np.log(z))[..., 0]).max() <= 1e-4
    args = (qf, kf, vf, f64(o), f64(lse), f64(do), None)
    want = O.attn_backward(*args, off, 1, fresh, scale)
    tol = bounds.backward(*args, O.selected_pairs(off, 1, fresh, N), scale, bounds.BF16)
    for n, x, w, e in zip(("dq", "dk", "dv"), out, want, tol):
        bounds.check(n, f64(x), w, e)


# ------------------------------------------------------------------ refusals
def test_length_outside_the_cache_is_clamped_and_reported(ctx):
    cache = make_cache(ctx, 2, 1, 100, 64, 12)
    q = queries(2, 1, 1, 64, "bf16", 12)
    ctx.sync_status()
    o, lse = attend(ctx, q, cache, starts([101, -5]))
    with pytest.raises(pa.PAError) as e:
        ctx.sync_status()
    assert e.value.code == -1
    compare(q, cache, [100, 0], o, lse, "bf16")


def test_refusals(ctx):
    cache = make_cache(ctx, 1, 2, 130, 64, 13)
    kc, vc, ks, vs = cache
    q = queries(1, 4, 1, 64, "bf16", 13)
    o, lse = torch.empty_like(q), torch.empty(1, 4, 1, device="cuda")
    lens = starts([100])

    def call(q=q, cache=cache, lens=lens, o=o, lse=lse, **kw):
        pa.pa_cache_attn(ctx, q, *cache, lens, o, lse, **kw)

    call()
    for kw in (dict(q=q.half()), dict(o=o.float()), dict(lse=lse.double()), dict(lens=lens.long()),
               dict(lens=starts([1, 2])), dict(q=q[0]), dict(cache=[kc.float(), vc, ks, vs]),
               dict(cache=[kc, vc[:, :, :64], ks, vs]), dict(cache=[kc, vc, ks[:, :, :2], vs]),
               dict(cache=[kc, vc, ks.cpu(), vs]), dict(lens=lens.cpu()), dict(scale=0.0),
               dict(scale=float("nan")), dict(q=queries(1, 3, 1, 64, "bf16", 0), o=queries(1, 3, 1, 64, "bf16", 0),
                                              lse=torch.empty(1, 3, 1, device="cuda"))):
        with pytest.raises(pa.PAError):
            call(**kw)
    long = make_cache(ctx, 1, 1, 5000, 64, 14)
    q1 = queries(1, 1, 1, 64, "bf16", 14)
    need = pa.cache_attn_workspace(ctx, q1, long[0]).numel()
    if need:
        with pytest.raises(pa.PAError):
            pa.pa_cache_attn(ctx, q1, *long, None, torch.empty_like(q1), torch.empty(1, 1, 1, device="cuda"),
                             workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    x = torch.zeros(1, 2, 5, 64, dtype=torch.bfloat16, device="cuda")
    for args in ((x, x.float(), None), (x, x[:, :, :4], None), (x.half(), x.half(), None), (x, x, lens.long()),
                 (x, x, starts([1, 2])), (x[:, :1], x[:, :1], None), (x[0], x[0], None)):
        with pytest.raises(pa.PAError):
            pa.pa_cache_store(ctx, *args, *cache)
    y = torch.zeros(1, 2, 131, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pa.PAError):
        pa.pa_cache_store(ctx, y, y, None, *cache)
    d96 = torch.zeros(1, 2, 130, 96, dtype=torch.uint8, device="cuda")
    q96 = torch.zeros(1, 2, 1, 96, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pa.PAError) as e:
        pa.pa_cache_attn(ctx, q96, d96, d96, ks, vs, None, q96, torch.empty(1, 2, 1, device="cuda"))
    assert e.value.code == -3
    call()
    ctx.sync_status()


def test_no_rows(ctx):
    cache = make_cache(ctx, 1, 1, 64, 64, 15)
    q = torch.empty(1, 2, 0, 64, dtype=torch.bfloat16, device="cuda")
    pa.pa_cache_attn(ctx, q, *cache, None, torch.empty_like(q), torch.empty(1, 2, 0, device="cuda"))
    x = torch.empty(1, 1, 0, 64, dtype=torch.bfloat16, device="cuda")
    pa.pa_cache_store(ctx, x, x, None, *cache)
    ctx.sync_status()
