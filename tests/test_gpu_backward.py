"""Backward pass of attention with reuse against the oracle, elementwise within the bounds of
the roundings made (tests/bounds.py)."""
import numpy as np
import pytest
import torch

import bounds
import oracle as O
import sequence_partition_attn_b200 as pa

pytestmark = pytest.mark.gpu
DT = {"f32": (torch.float32, bounds.F32), "bf16": (torch.bfloat16, bounds.BF16)}


@pytest.fixture(scope="module")
def ctx():
    c = pa.Context(0)
    yield c
    c.close()


def f64(t):
    return t.detach().double().cpu().numpy()


def make(B, H, N, D, dtype, off, G, fresh, seed, dlse=False, gain=1.0):
    """Inputs on the device and the merged forward outputs (all pairs, so that o and lse hold
    pairs that the mask does not select, as reused states would)."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype][0]
    q, k, v, do = (torch.randn(B, H, N, D, generator=g).mul(gain if i < 2 else 1.0).to(dt) for i in range(4))
    scale = D ** -0.5
    s = scale * np.einsum("bhid,bhjd->bhij", f64(q), f64(k))
    m = s.max(-1, keepdims=True)
    z = np.exp(s - m).sum(-1, keepdims=True)
    o = torch.from_numpy(np.einsum("bhij,bhjd->bhid", np.exp(s - m) / z, f64(v))).to(dt)
    lse = torch.from_numpy((m + np.log(z))[..., 0]).float()
    dl = torch.randn(B, H, N, generator=g) if dlse else None
    t = dict(q=q, k=k, v=v, o=o, lse=lse, do=do, dlse=dl)
    return {n: None if x is None else x.cuda() for n, x in t.items()}


def grads(ctx, t, off, G, fresh, scale=None, stream=None):
    out = [torch.full_like(t["q"], float("nan")) for _ in range(3)]
    delta = torch.full_like(t["lse"], float("nan"))
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())          # which fills the outputs
    pa.pa_attn_backward(ctx, t["q"], t["k"], t["v"], t["o"], t["lse"], t["do"], off, G, fresh, *out, delta,
                        dlse=t["dlse"], scale=scale, stream=stream)
    return out, delta


def compare(t, out, delta, off, G, fresh, dtype, scale=None):
    D, N = t["q"].shape[3], t["q"].shape[2]
    scale = D ** -0.5 if scale is None else scale
    a = {n: None if x is None else f64(x) for n, x in t.items()}
    args = (a["q"], a["k"], a["v"], a["o"], a["lse"], a["do"], a["dlse"])
    want = O.attn_backward(*args, off, G, fresh, scale)
    tol = bounds.backward(*args, O.selected_pairs(off, G, fresh, N), scale, DT[dtype][1])
    for n, x, w, e in zip(("dq", "dk", "dv"), out, want, tol):
        bounds.check(n, f64(x), w, e)
    mag = (np.abs(a["do"]) * np.abs(a["o"])).sum(-1) + (0 if a["dlse"] is None else np.abs(a["dlse"]))
    bounds.check("delta", f64(delta), want[3], 2 * (D + 1) * bounds.U * mag + 1e-37)


def even(N, P):
    S = -(-N // P)
    return np.array([min(p * S, N) for p in range(P + 1)])


CASES = [
    # B, H, N, D, P offsets, G, mask density (1 = NULL mask)
    (1, 1, 1, 64, [0, 1], 1, 1),
    (1, 2, 2, 128, [0, 1, 2], 1, 0.6),
    (1, 1, 63, 64, [0, 63], 1, 1),
    (1, 1, 64, 128, [0, 64], 1, 1),
    (2, 1, 65, 64, [0, 32, 65], 1, 0.6),
    (1, 1, 127, 128, [0, 127], 1, 1),
    (1, 2, 128, 64, [0, 128], 1, 1),
    (1, 1, 129, 128, [0, 128, 129], 1, 0.7),
    (1, 1, 255, 64, [0, 0, 100, 100, 255, 255], 2, 0.6),
    (1, 1, 256, 128, [0, 16, 17, 150, 256], 1, 0.5),
    (2, 2, 333, 128, None, 3, 0.5),
    (1, 3, 640, 64, None, 1, 0.4),
    (1, 1, 1000, 128, None, 2, 1),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_formulas(ctx, case, dtype):
    B, H, N, D, off, G, density = CASES[case]
    off = even(N, 9) if off is None else np.array(off)
    QG = -(-(len(off) - 1) // G)
    rng = np.random.default_rng(case)
    fresh = None if density == 1 else (rng.random((QG, QG)) < density).astype(np.uint8)
    t = make(B, H, N, D, dtype, off, G, fresh, 10 + case, dlse=case % 2 == 0)
    out, delta = grads(ctx, t, off, G, fresh)
    ctx.sync_status()
    compare(t, out, delta, off, G, fresh, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_groups_without_a_fresh_pair_get_zeros(ctx, dtype):
    off = even(500, 5)
    fresh = np.zeros((5, 5), dtype=np.uint8)
    fresh[1, 3] = fresh[2, 3] = 1
    t = make(1, 2, 500, 64, dtype, off, 1, fresh, 3)
    out, delta = grads(ctx, t, off, 1, fresh)
    compare(t, out, delta, off, 1, fresh, dtype)
    assert not out[0][:, :, :100].any() and not out[0][:, :, 300:].any()
    for x in out[1:]:
        assert not x[:, :, :300].any() and not x[:, :, 400:].any()
    out, _ = grads(ctx, t, off, 1, np.zeros((5, 5), dtype=np.uint8))
    assert not any(x.any() for x in out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [5, 150])
def test_rows_of_other_pairs_may_hold_anything(ctx, dtype, width):
    """Infinities and NaN in every row that no fresh pair holds leave the gradients alone."""
    N, D = 600, 128
    off = np.array([0, 200, 200 + width, 500, N])
    fresh = np.zeros((4, 4), dtype=np.uint8)
    fresh[1, 1] = 1
    t = make(1, 1, N, D, dtype, off, 1, fresh, 4)
    out, _ = grads(ctx, t, off, 1, fresh)
    for n in ("q", "k", "v", "o", "do"):
        for sl in (slice(0, 200), slice(200 + width, N)):
            t[n][:, :, sl, ::2] = float("nan")
            t[n][:, :, sl, 1::2] = float("inf")
    t["lse"][:, :, :200] = float("nan")
    t["lse"][:, :, 200 + width:] = float("nan")
    dirty, _ = grads(ctx, t, off, 1, fresh)
    for a, b in zip(out, dirty):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_without_keys(ctx, dtype):
    """lse = -inf (no key at all) means every probability is 0."""
    off = even(300, 3)
    t = make(1, 2, 300, 64, dtype, off, 1, None, 5, dlse=True)
    t["lse"][:, :, 17:40] = float("-inf")
    out, delta = grads(ctx, t, off, 1, None)
    assert not out[0][:, :, 17:40].any()
    compare(t, out, delta, off, 1, None, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gain", [1e-3, 6.0])
def test_flat_and_peaked_probabilities(ctx, dtype, gain):
    off = even(300, 2)
    t = make(1, 2, 300, 128, dtype, off, 1, None, 6, gain=gain)
    out, delta = grads(ctx, t, off, 1, None)
    compare(t, out, delta, off, 1, None, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_own_scale_and_repeatability(ctx, dtype):
    off = even(700, 4)
    t = make(1, 2, 700, 64, dtype, off, 2, None, 7)
    t["lse"] = t["lse"] + 1.0                       # a scale other than the inputs' needs only P <= 1
    a, delta = grads(ctx, t, off, 2, None, scale=0.05)
    compare(t, a, delta, off, 2, None, dtype, scale=0.05)
    b, _ = grads(ctx, t, off, 2, None, scale=0.05)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradient_matches_differences_of_the_forward_path(ctx):
    """f32: d/dx of <do, o> + <dlse, lse> through pa_partition_attn + pa_merge_states with
    cached states, by central differences along random directions."""
    B, H, N, D, G = 1, 2, 96, 64, 1
    off = np.array([0, 20, 53, N])
    fresh = np.array([[1, 0, 1], [1, 1, 0], [0, 0, 1]], dtype=np.uint8)
    g = torch.Generator().manual_seed(8)
    q, k, v, do = (torch.randn(B, H, N, D, generator=g).cuda() for _ in range(4))
    dlse = torch.randn(B, H, N, generator=g).cuda()
    P = 3
    oc, lc = torch.empty(P, B, H, N, D, device="cuda"), torch.empty(P, B, H, N, device="cuda")
    pa.pa_partition_attn(ctx, q, k * 1.1, v * 0.9, off, G, None, oc, lc)

    def forward(q, k, v):
        of, lf = torch.zeros_like(oc), torch.zeros_like(lc)
        pa.pa_partition_attn(ctx, q, k, v, off, G, fresh, of, lf)
        o, lse = torch.empty_like(q), torch.empty(B, H, N, device="cuda")
        pa.pa_merge_states(ctx, off, G, fresh, of, lf, oc, lc, o, lse)
        return o, lse

    o, lse = forward(q, k, v)
    t = dict(q=q, k=k, v=v, o=o, lse=lse, do=do, dlse=dlse)
    out, _ = grads(ctx, t, off, G, fresh)
    loss = lambda o, l: float((o.double() * do.double()).sum() + (l.double() * dlse.double()).sum())  # noqa: E731
    eps = 2.0 ** -7
    for i in range(3):
        for seed in range(3):
            d = torch.randn(B, H, N, D, generator=torch.Generator().manual_seed(100 + seed)).cuda()
            hi = [x + eps * d if j == i else x for j, x in enumerate((q, k, v))]
            lo = [x - eps * d if j == i else x for j, x in enumerate((q, k, v))]
            diff = (loss(*forward(*hi)) - loss(*forward(*lo))) / (2 * eps)
            want = float((out[i].double() * d.double()).sum())
            # Third-order term: eps^2 / 6 times the third derivative along d.  The scores move by
            # sigma = |scale q.d| ~ 1 per unit and the loss's terms sum B H N (D + 1) products of
            # unit size, so it is about eps^2 sqrt(B H N (D + 1)) (1e-2); fp32 noise of the loss
            # difference is 2^-24 times the same sum's 12480 terms / (2 eps): below 5e-2.
            assert abs(diff - want) <= 0.1 + 2e-3 * abs(want), (i, seed, diff, want)


def test_other_stream_and_graph_replay(ctx):
    off = even(520, 4)
    t = make(1, 2, 520, 128, "bf16", off, 1, None, 9)
    a, _ = grads(ctx, t, off, 1, None)
    s = torch.cuda.Stream()
    b, _ = grads(ctx, t, off, 1, None, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    out = [torch.zeros_like(t["q"]) for _ in range(3)]
    delta = torch.zeros_like(t["lse"])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pa.pa_attn_backward(ctx, t["q"], t["k"], t["v"], t["o"], t["lse"], t["do"], off, 1, None, *out, delta)
    t["do"].mul_(2.0)                                # the replay reads the tensors of then
    graph.replay()
    torch.cuda.synchronize()
    want, _ = grads(ctx, t, off, 1, None)
    assert all(torch.equal(x, y) for x, y in zip(out, want))
    ctx.sync_status()


def test_two_streams_at_once(ctx):
    off = even(900, 3)
    ts = [make(1, 3, 900, 64, "bf16", off, 1, None, 20 + i) for i in range(2)]
    want = [grads(ctx, t, off, 1, None)[0] for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(3):
        # both deltas stay allocated until the streams are done with them
        got = [grads(ctx, t, off, 1, None, stream=s) for t, s in zip(ts, streams)]
        torch.cuda.synchronize()
        for a, (b, _) in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals(ctx):
    off = even(64, 2)
    t = make(1, 1, 64, 64, "bf16", off, 1, None, 1)
    ok = [t["q"], t["k"], t["v"], t["o"], t["lse"], t["do"]]
    out = [torch.empty_like(t["q"]) for _ in range(3)]
    delta = torch.empty_like(t["lse"])

    def call(args=ok, off=off, G=1, fresh=None, out=out, delta=delta, **kw):
        pa.pa_attn_backward(ctx, *args, off, G, fresh, *out, delta, **kw)

    call()
    bad = t["k"].float()
    with pytest.raises(pa.PAError):
        call(args=[t["q"], bad, *ok[2:]])
    with pytest.raises(pa.PAError):
        call(args=[t["q"].half(), *ok[1:]])
    with pytest.raises(pa.PAError):
        call(args=[t["q"], t["k"][:, :, :32], *ok[2:]])
    wide = torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pa.PAError):                 # a view with strides of its own
        call(args=[t["q"], wide[..., ::2], *ok[2:]])
    with pytest.raises(pa.PAError):
        call(args=[t["q"], t["k"].cpu(), *ok[2:]])
    with pytest.raises(pa.PAError):
        call(delta=delta.double())
    with pytest.raises(pa.PAError):
        call(dlse=delta[:, :, :3])
    for o in ([0, 10], [1, 64], [0, 65], [0, 40, 30, 64]):
        with pytest.raises(pa.PAError):
            call(off=o)
    for G in (0, 3):
        with pytest.raises(pa.PAError):
            call(G=G)
    with pytest.raises(pa.PAError):
        call(fresh=np.ones((3, 3), dtype=np.uint8))
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(pa.PAError):
            call(scale=scale)
    flat = torch.zeros(64 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(1, 1, 64, 64)
    with pytest.raises(pa.PAError) as e:
        call(args=[flat, *ok[1:]])
    assert e.value.code == -2
    d96 = [torch.zeros(1, 1, 64, 96, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    with pytest.raises(pa.PAError) as e:
        pa.pa_attn_backward(ctx, *d96[:4], t["lse"], d96[4], off, 1, None, *d96[5:], delta)
    assert e.value.code == -3
    call()
    ctx.sync_status()


def test_no_rows(ctx):
    z = [torch.empty(1, 2, 0, 64, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    r = torch.empty(1, 2, 0, device="cuda")
    pa.pa_attn_backward(ctx, *z[:4], r, z[4], [0, 0], 1, None, *z[5:], r)
    ctx.sync_status()
