"""Host side of the backward pass and the 8-bit cache (no GPU needed): the oracle against
definitions of its own, and arguments that the binding refuses before any launch."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import oracle as O
import sequence_partition_attn_b200 as pa
from sequence_partition_attn_b200 import build as pa_build


def forward(q, k, v, off, G, fresh, lc, oc, scale):
    """Merged output of the fresh pairs and one constant state (oc, lc) per row."""
    sel = O.selected_pairs(off, G, fresh, q.shape[2])
    s = np.where(sel, scale * np.einsum("bhid,bhjd->bhij", q, k), -np.inf)
    e, ec = np.exp(s), np.exp(lc)
    z = e.sum(-1) + ec
    return (np.einsum("bhij,bhjd->bhid", e, v) + ec[..., None] * oc) / z[..., None], np.log(z)


@pytest.mark.parametrize("G,fresh", [(1, None), (1, [[1, 0, 1], [0, 0, 0], [1, 1, 0]]), (2, [[0, 1], [1, 1]])])
def test_oracle_gradient_matches_differences(G, fresh):
    rng = np.random.default_rng(0)
    B, H, N, D, scale = 1, 2, 7, 5, 0.4
    off = np.array([0, 2, 2 if G == 2 else 4, N])
    q, k, v, do, oc = (rng.standard_normal((B, H, N, D)) for _ in range(5))
    lc, dlse = rng.standard_normal((B, H, N)), rng.standard_normal((B, H, N))
    o, lse = forward(q, k, v, off, G, fresh, lc, oc, scale)
    got = O.attn_backward(q, k, v, o, lse, do, dlse, off, G, fresh, scale)
    np.testing.assert_allclose(got[3], (do * o).sum(-1) - dlse)
    x, eps = [q, k, v], 1e-5
    for i in range(3):
        num = np.zeros_like(q)
        for at in np.ndindex(q.shape):
            val = []
            for sgn in (1, -1):
                y = [a.copy() for a in x]
                y[i][at] += sgn * eps
                oo, ll = forward(*y, off, G, fresh, lc, oc, scale)
                val.append((oo * do).sum() + (ll * dlse).sum())
            num[at] = (val[0] - val[1]) / (2 * eps)
        np.testing.assert_allclose(got[i], num, atol=1e-8)


def test_e4m3_rounding_matches_torch_and_its_own_values():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    vals = codes[~codes.isnan()].double().numpy()
    np.testing.assert_array_equal(O.e4m3_round(vals), vals)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 6, 4000),
                        (vals[1:] + vals[:-1]) / 2]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().double().numpy()
    np.testing.assert_array_equal(O.e4m3_round(x), want)
    assert O.e4m3_round(np.inf) == 448 and np.isnan(O.e4m3_round(np.nan))


def test_cache_scale_is_the_smallest_power_of_two():
    for e in range(-110, 110, 7):
        for f in (1.0, 1.3, 1.75, np.nextafter(1.75, 2), 1.99):
            a = f * 2.0 ** e
            s = O.cache_scale(a)
            assert a <= 448 * s and (a > 448 * s / 2)
    assert O.cache_scale(0.0) == 0.0 and O.cache_scale(1e-45) == 2.0 ** -126


def test_oracle_cache_attention_is_softmax_over_the_held_tokens():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((2, 4, 3, 8)), rng.standard_normal((2, 2, 9, 8)), rng.standard_normal((2, 2, 9, 8))
    o, lse = O.cache_attn(q, k, v, [9, 4], 0.3)
    tq, tk, tv = (torch.from_numpy(x) for x in (q, k, v))
    for b, n in enumerate((9, 4)):
        kk, vv = (x[b, :, :n].repeat_interleave(2, dim=0) for x in (tk, tv))
        s = 0.3 * tq[b] @ kk.transpose(1, 2)
        np.testing.assert_allclose(o[b], (s.softmax(-1) @ vv).numpy(), atol=1e-12)
        np.testing.assert_allclose(lse[b], s.logsumexp(-1).numpy(), atol=1e-12)
    o, lse = O.cache_attn(q, k, v, [0, 9], 0.3)
    assert not o[0].any() and np.isneginf(lse[0]).all()


# ------------------------------------------------------------------ refusals before any launch
@pytest.fixture(scope="module")
def fake_ctx():
    pa_build.build()
    return SimpleNamespace(ptr=None, device=0)


def test_null_context_is_rejected(fake_ctx):
    L = pa.lib()
    assert L.pa_attn_backward(None, None, None) == -1
    assert L.pa_cache_store(None, None, None) == -1
    assert L.pa_cache_attn(None, None, None) == -1
    assert L.pa_cache_attn_ws(None, 1, 1, 1, 1, 1, 1, 64, None) == -1


def test_host_tensors_and_bad_masks_are_rejected(fake_ctx):
    z = [torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16) for _ in range(8)]
    r = torch.zeros(1, 1, 8)
    args = (*z[:4], r, z[4])
    with pytest.raises(pa.PAError, match="is on cpu"):
        pa.pa_attn_backward(fake_ctx, *args, [0, 8], 1, None, *z[5:], r, stream=0)
    for off, G, fresh in (([0], 1, None), ([0, 8], 0, None), ([0, 8], 2, None), ([0, 4, 8], 1, np.ones((3, 3)))):
        with pytest.raises(pa.PAError):
            pa.pa_attn_backward(fake_ctx, *args, off, G, fresh, *z[5:], r, stream=0)
    kc = torch.zeros(1, 1, 8, 64, dtype=torch.uint8)
    s = torch.zeros(1, 1, 1)
    with pytest.raises(pa.PAError, match="is on cpu"):
        pa.pa_cache_store(fake_ctx, z[0], z[1], None, kc, kc, s, s, stream=0)
    with pytest.raises(pa.PAError, match="is on cpu"):
        pa.pa_cache_attn(fake_ctx, z[0], kc, kc, s, s, None, z[1], r, stream=0)
    with pytest.raises(pa.PAError, match="dtype"):
        pa.pa_cache_attn(fake_ctx, z[0], kc.float(), kc, s, s, None, z[1], r, stream=0)
