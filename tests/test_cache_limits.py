"""The 8-bit cache at the ends of its sizes, and a request alone and in a batch."""
import pytest
import torch

import bounds
import oracle as O
import sequence_partition_attn_b200 as pa
from test_gpu_cache import DT, attend, f64, make_cache, queries, starts, values

pytestmark = pytest.mark.gpu


def test_token_counts_near_the_end_of_32_bits_are_refused():
    """Kernels count tokens in 32 bits, past a request's last one by up to a tile.  T = 0: nothing
    would run in any case."""
    ctx = pa.Context(0)
    for M, want in ((2 ** 31 - 1, -1), (2 ** 31 - 1024, -1), (2 ** 31 - 1025, 0)):
        desc = pa._CACHE_STORE.pack(pa.PA_BF16, 1, 1, 0, M, 64, 0, 0, 0, 0, 0, 0, 0)
        assert pa.lib().pa_cache_store(ctx.ptr, desc, 0) == want, M
        desc = pa._CACHE_ATTN.pack(pa.PA_BF16, 1, 1, 1, 0, M, 64, 0.125, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
        assert pa.lib().pa_cache_attn(ctx.ptr, desc, 0) == want, M
    ctx.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Nq", [1, 5, 60])
def test_a_request_alone_and_in_a_batch(dtype, Nq):
    """The cuts of the work follow the whole batch, so the bits may differ; both are within the bound of
    the roundings.  Repeated, either gives the same bits."""
    ctx = pa.Context(0)
    B, H, Hk, M, D = 5, 8, 4, 2000, 128
    lens = [2000, 450, 1, 0, 1999]
    cache = make_cache(ctx, B, Hk, M, D, 70)
    q = queries(B, H, Nq, D, dtype, 70)
    batch = attend(ctx, q, cache, starts(lens))
    k, v = values(cache)
    want = O.cache_attn(f64(q), k, v, lens, D ** -0.5)
    tol = bounds.attention(f64(q), k, v, lens, D ** -0.5, DT[dtype][1])
    for b, n in enumerate(lens):
        one = [x[b:b + 1].contiguous() for x in cache]
        alone = attend(ctx, q[b:b + 1].contiguous(), one, starts([n]))
        again = attend(ctx, q[b:b + 1].contiguous(), one, starts([n]))
        assert all(torch.equal(x, y) for x, y in zip(alone, again))
        for got in (alone, [x[b:b + 1] for x in batch]):
            bounds.check("o", f64(got[0]), want[0][b:b + 1], tol[0][b:b + 1])
            bounds.check("lse", f64(got[1]), want[1][b:b + 1], tol[1][b:b + 1])
    assert all(torch.equal(x, y) for x, y in zip(batch, attend(ctx, q, cache, starts(lens))))
    ctx.sync_status()
    ctx.close()
