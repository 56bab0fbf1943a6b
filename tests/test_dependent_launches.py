"""Kernels that are launched ahead of the end of the one before them (programmatic serialisation).

What follows such a kernel in a stream or a graph is ordered behind it alone, so it has to wait for
its predecessor on every path, results of its own to write or not.
"""
import os
import re

import numpy as np
import pytest
import torch

import sequence_partition_attn_b200 as pa

CSRC = os.path.join(os.path.dirname(os.path.abspath(pa.__file__)), "csrc")


def test_the_join_waits_before_its_first_return():
    """A row that one piece covered has nothing to join.  With every request inside one cache block
    that is every row: if they returned first, no thread of the grid would wait."""
    src = open(os.path.join(CSRC, "cache_attn_rows.cu")).read()
    body = re.search(r"cache_attn_rows_join_kernel\(const __grid_constant__.*?\n}\n", src, re.S).group(0)
    body = re.sub(r"//[^\n]*", "", body)
    assert body.index("griddepcontrol.wait") < body.index("return")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,Hk,M,longest", [(64, 24, 24, 4096, 64), (1, 8, 8, 4096, 100), (7, 6, 2, 640, 128), (300, 8, 8, 1024, 1)])
def test_a_graph_reads_the_state_behind_the_call(B, H, Hk, M, longest, dtype):
    """Caches with room for more than they hold: no unit is cut, and the next nodes of the graph
    use o and lse at once.  The queries change between replays."""
    D = 128
    ctx = pa.Context(0)
    g = torch.Generator().manual_seed(B)
    nb = -(-M // pa.PA_CACHE_BLOCK)
    cache = [torch.zeros(B, Hk, M, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.zeros(B, Hk, nb, device="cuda") for _ in range(2)]
    rows = [torch.randn(B, Hk, longest, D, generator=g).cuda() for _ in range(2)]
    pa.pa_cache_store(ctx, *rows, None, *cache)
    held = np.random.default_rng(B).integers(1, longest + 1, B).astype(np.int32)
    lens = torch.from_numpy(held).cuda()
    qs = [torch.randn(B, H, 1, D, generator=g).to(dtype).cuda() for _ in range(3)]
    q, o, lse = qs[0].clone(), torch.zeros_like(qs[0]), torch.zeros(B, H, 1, device="cuda")
    ws = pa.cache_attn_workspace(ctx, q, cache[0])
    assert ws.numel() > 0                                       # the form that joins
    want = []
    for x in qs:
        q.copy_(x)
        pa.pa_cache_attn(ctx, q, *cache, lens, o, lse, workspace=ws)
        torch.cuda.synchronize()
        want.append((o.clone(), lse.clone()))
    got = [(torch.zeros_like(o), torch.zeros_like(lse)) for _ in qs]
    seen = [torch.zeros_like(o), torch.zeros_like(lse)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_cache_attn(ctx, q, *cache, lens, o, lse, workspace=ws)
        seen[0].copy_(o)
        seen[1].copy_(lse)
        o.zero_()                                               # a late store would show next time
        lse.zero_()
    for _ in range(4):
        for x, y in zip(qs, got):
            q.copy_(x)
            graph.replay()
            for a, b in zip(y, seen):
                a.copy_(b)
        torch.cuda.synchronize()
        for y, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(y, w))
    ctx.sync_status()
    ctx.close()
