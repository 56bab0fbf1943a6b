"""Sizes at the ends of what the 8-bit cache takes."""
import pytest

import sequence_partition_attn_b200 as pa

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
