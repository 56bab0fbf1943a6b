"""The backward pass's scratch of an attention step: allocated by the first backward pass."""
import contextlib
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import sequence_partition_attn_b200 as pa
from sequence_partition_attn_b200 import step as step_module
from sequence_partition_attn_b200.step import AttentionStep


def test_a_step_without_a_backward_pass_holds_no_scratch_for_one(monkeypatch):
    seen, current = [], SimpleNamespace(stream=0x70)

    @contextlib.contextmanager
    def on(s):
        before, current.stream = current.stream, s.cuda_stream
        yield
        current.stream = before

    def backward(ctx, q, k, v, o, lse, do, off, G, fresh, dq, dk, dv, delta, dlse=None, stream=None):
        seen.append(delta)

    real = torch.empty_like
    allocated = []
    monkeypatch.setattr(torch, "empty_like", lambda t: allocated.append(current.stream) or real(t))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device=None: SimpleNamespace(cuda_stream=s))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: current.stream, raising=False)
    monkeypatch.setattr(step_module, "pa_attn_backward", backward)
    step = AttentionStep(SimpleNamespace(device=0), 1, 2, 10, 64, [0, 5, 10], 1, None, device="cpu")
    assert step.delta is None
    g = [torch.zeros(1, 2, 10, 64) for _ in range(4)]
    step.backward(*g, stream=0x50)
    step.backward(*g)
    assert allocated == [0x50]                                  # for the stream that the first one runs on
    assert seen[0] is seen[1] is step.delta
    assert step.delta.shape == (1, 2, 10) and step.delta.dtype == torch.float32


@pytest.mark.gpu
def test_first_backward_pass_in_a_graph():
    """The scratch outlives the graph that it was allocated in."""
    ctx = pa.Context(0)
    B, H, N, D = 1, 2, 300, 64
    step = AttentionStep(ctx, B, H, N, D, np.array([0, 100, N]), 1, None)
    for n in ("q", "k", "v"):
        getattr(step, n).copy_(torch.randn(B, H, N, D, generator=torch.Generator().manual_seed(len(n) + ord(n[0]))))
    step.run()
    do = torch.randn(B, H, N, D, generator=torch.Generator().manual_seed(9)).to(step.q)
    got, want = ([torch.zeros_like(step.q) for _ in range(3)] for _ in range(2))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.backward(do, *got)
    graph.replay()
    torch.cuda.synchronize()
    held = step.delta
    del graph
    junk = [torch.full((B, H, N), float("nan"), device="cuda") for _ in range(8)]
    step.backward(do, *want)
    ctx.sync_status()
    assert step.delta is held
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool(torch.isnan(x).all()) for x in junk)
    ctx.close()
