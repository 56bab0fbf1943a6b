"""Sums over a long token axis in the fp32 form of pa_cache_attn."""
import pytest
import torch

import bounds
import sequence_partition_attn_b200 as pa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [False, True])
def test_fp32_sums_are_rounded_and_not_cut(D, far):
    """So many rows that a block of threads walks all tokens for each 8 of them, and values above
    zero, whose sum grows: an error of one sign for each addition would be seen.

    One channel of q is set, so a score is one product, exact in fp32.  A weight errs by the
    exponential (2^-22), its argument (three roundings of |s| < 8, in natural units 24 u) and its two
    terms (2^-23): below 2^-20 with that of the sum that divides it.  A running sum takes one addition per
    64 tokens and warp; rounded additions err by u each and either sign, so that n of them stay within
    6 sqrt(n) u (six standard deviations, were every one of full size).  Cut ones err by n u / 2.
    `far`: the same with blocks of V 2^-20 apart, of which the small ones take the other form of product."""
    M, rows = 65536, 8 * 500
    ctx = pa.Context(0)
    g = torch.Generator(device="cuda").manual_seed(D)
    k = torch.randn(1, 1, M, D, generator=g, device="cuda")
    v = 1.0 + 0.5 * torch.rand(1, 1, M, D, generator=g, device="cuda")
    if far:
        v[:, :, 64:] *= 2.0 ** -20                              # one block far above all others,
        k[:, :, :64, 0] = -60.0                                 # without weight
    kc, vc = (torch.empty(1, 1, M, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(1, 1, M // 64, device="cuda") for _ in range(2))
    pa.pa_cache_store(ctx, k, v, None, kc, vc, ks, vs)
    q = torch.zeros(1, 1, rows, D, device="cuda")
    q[..., 0] = torch.rand(rows, generator=g, device="cuda") + 0.5
    o, lse = torch.empty_like(q), torch.empty(1, 1, rows, device="cuda")
    pa.pa_cache_attn(ctx, q, kc, vc, ks, vs, None, o, lse, scale=1.0)
    ctx.sync_status()
    kk, vv = (c[0, 0].view(torch.float8_e4m3fn).double() * s[0, 0].double().repeat_interleave(64)[:, None]
              for c, s in ((kc, ks), (vc, vs)))
    assert float(kk[64:, 0].abs().max()) * 1.5 < 8
    n = M // 64
    tol = 2.0 ** -20 + 6 * n ** 0.5 * bounds.U
    for r in range(0, rows, 250):
        s = q[0, 0, r].double() @ kk.T
        want = torch.softmax(s, 0) @ vv
        err = (o[0, 0, r].double() - want).abs() / want
        assert float(err.max()) <= tol, (r, float(err.max()), tol)
        assert abs(float(lse[0, 0, r]) - float(torch.logsumexp(s, 0))) <= tol + 4 * bounds.U * 12
    ctx.close()


def test_bf16_sums_over_a_million_tokens():
    """So many rows that the token axis need not be cut to fill the GPU.  The tensor cores cut their sums
    by up to 2^-23 for each 16 tokens; a chain of them is at most 131072 tokens long: 2^13 steps, 2^-10
    of O.  The mean over the channels shows it under the output's rounding (2^-8, either sign, six
    standard deviations of 64 uniform errors); flat scores, so that the weights' rounding averages out.
    lse: a score errs by 2 D u sum|scale q k| (0.5), a sum of 1024 tiles by 6 sqrt(1024) u, the result by
    4 u 14: below 2^-15 together."""
    D, M, rows = 64, 1 << 20, 256 * 150
    ctx = pa.Context(0)
    g = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.empty(1, 1, M, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(1, 1, M // 64, device="cuda") for _ in range(2))
    k = torch.randn(1, 1, M, D, generator=g, device="cuda")
    v = 1.0 + 0.9 * torch.rand(1, 1, M, D, generator=g, device="cuda")
    v *= 1.0 + torch.arange(D, device="cuda") / D               # channels whose roundings are not alike
    pa.pa_cache_store(ctx, k, v, None, kc, vc, ks, vs)
    q = torch.randn(1, 1, rows, D, generator=g, device="cuda").mul_(0.1).to(torch.bfloat16)
    o, lse = torch.full_like(q, float("nan")), torch.full((1, 1, rows), float("nan"), device="cuda")
    pa.pa_cache_attn(ctx, q, kc, vc, ks, vs, None, o, lse)
    ctx.sync_status()
    kk, vv = (c[0, 0].view(torch.float8_e4m3fn).double() * s[0, 0].double().repeat_interleave(64)[:, None]
              for c, s in ((kc, ks), (vc, vs)))
    tol = 2.0 ** -10 + 6 * 2.0 ** -8 / (3 * D) ** 0.5 + 2.0 ** -15
    for r in range(0, rows, 2500):
        s = D ** -0.5 * (q[0, 0, r].double() @ kk.T)
        want = torch.softmax(s, 0) @ vv
        err = (o[0, 0, r].double() - want) / want
        assert abs(float(err.mean())) <= tol, (r, float(err.mean()), tol)
        assert float(err.abs().max()) <= 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -15
        assert abs(float(lse[0, 0, r]) - float(torch.logsumexp(s, 0))) <= 2.0 ** -15
    ctx.close()
