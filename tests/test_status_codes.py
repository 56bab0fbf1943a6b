"""The context's status word: what kernels record there and what pa_sync_status makes of it."""
import glob
import os
import re

import pytest
import torch

import sequence_partition_attn_b200 as pa

CSRC = os.path.join(os.path.dirname(os.path.abspath(pa.__file__)), "csrc")


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["store", "attend"])
@pytest.mark.parametrize("order", ["before", "behind"])
def test_a_wait_that_gave_up_outweighs_a_bad_length(call, order):
    """Both happen before the status is read: a time-out means that results are missing, so it is
    the one reported, once."""
    ctx = pa.Context(0)
    kc, vc = (torch.zeros(1, 1, 64, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(1, 1, 1, device="cuda") for _ in range(2))
    x, o = (torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    outside = torch.tensor([65], dtype=torch.int32, device="cuda")

    def bad():
        if call == "store":
            pa.pa_cache_store(ctx, x, x, outside, kc, vc, ks, vs)
        else:
            pa.pa_cache_attn(ctx, x, kc, vc, ks, vs, outside, o, torch.empty(1, 1, 1, device="cuda"))

    if order == "before":
        bad()
    pa.pa_selftest_wait(ctx, 0.02)
    if order == "behind":
        bad()
    with pytest.raises(pa.PAError, match="PA_ETIMEOUT"):
        ctx.sync_status()
    ctx.sync_status()
    bad()
    with pytest.raises(pa.PAError, match="PA_EINVAL"):
        ctx.sync_status()
    ctx.close()


def test_every_recorded_code_is_reported_as_itself():
    recorded = set()
    for path in glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")):
        recorded |= set(re.findall(r"record_status\([^;]*\b(PA_E\w+)\)", open(path).read()))
    assert recorded >= {"PA_ETIMEOUT", "PA_EINVAL"}
    read = re.search(r"static int read_status\(.*?\n}\n", open(os.path.join(CSRC, "pa_abi.cu")).read(), re.S).group(0)
    assert recorded == set(re.findall(r"h == (PA_E\w+)\) return fail\(ctx, \1,", read))
