"""The scratch that pa_cache_attn takes itself belongs to the stream that uses it.

The allocator hands freed memory out again to the stream it was allocated for without waiting: that
is safe only for work on this stream.
"""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import sequence_partition_attn_b200 as pa


class FakeTensor(SimpleNamespace):
    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def record_stream(self, stream):
        pass


CURRENT = 0x70


@pytest.fixture
def host(monkeypatch):
    """The binding without a GPU: which stream was current when scratch was allocated, and which
    stream the call was given."""
    seen = SimpleNamespace(current=CURRENT, allocated=[], called=[])

    @contextlib.contextmanager
    def stream(s):
        before, seen.current = seen.current, s.cuda_stream
        yield
        seen.current = before

    def empty(n, dtype=None, device=None):
        seen.allocated.append(seen.current)
        return FakeTensor(shape=(n,), dtype=dtype, device=device)

    def ws(ptr, dtype, B, H, Hk, Nq, M, D, size):
        size._obj.value = 4096
        return 0

    def attn(ptr, desc, s):
        seen.called.append(s)
        return 0

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device=None: SimpleNamespace(cuda_stream=s))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: seen.current, raising=False)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(pa, "lib", lambda: SimpleNamespace(pa_cache_attn_ws=ws, pa_cache_attn=attn))
    return seen


def call(**kw):
    ctx = SimpleNamespace(ptr=1, _ptr=1, device=0)
    q, o = (FakeTensor(shape=(1, 2, 1, 64), dtype=torch.bfloat16) for _ in range(2))
    codes = FakeTensor(shape=(1, 1, 1000, 64), dtype=torch.uint8)
    scale = FakeTensor(shape=(1, 1, 16), dtype=torch.float32)
    pa.pa_cache_attn(ctx, q, codes, codes, scale, scale, None, o, FakeTensor(shape=(1, 2, 1), dtype=torch.float32), **kw)


@pytest.mark.parametrize("given", ["none", "current", "handle", "stream", "default handle"])
def test_scratch_is_allocated_for_the_stream_of_the_call(host, given):
    stream = {"none": None, "current": CURRENT, "handle": 0x50, "stream": SimpleNamespace(cuda_stream=0x60),
              "default handle": 0}[given]
    want = {"none": CURRENT, "current": CURRENT, "handle": 0x50, "stream": 0x60, "default handle": 0}[given]
    call(stream=stream)
    assert host.called == [want] and host.allocated == [want]
    assert host.current == CURRENT


def test_no_scratch_is_allocated_beside_the_given_one(host):
    call(workspace=FakeTensor(shape=(4096,), dtype=torch.uint8), stream=0x50)
    assert host.called == [0x50] and host.allocated == []


@pytest.mark.gpu
@pytest.mark.parametrize("handle", ["side", "default"])
def test_memory_in_use_on_the_current_stream_is_not_taken_for_another(handle):
    """Memory freed on the current stream behind work that still reads it, then a call on another
    stream: the reader finds what it was given, and the state is right."""
    B, Hk, M, D = 2, 8, 4096, 128
    ctx = pa.Context(0)
    g = torch.Generator().manual_seed(1)
    cache = [torch.empty(B, Hk, M, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache += [torch.empty(B, Hk, M // 64, device="cuda") for _ in range(2)]
    rows = [torch.randn(B, Hk, M, D, generator=g).cuda() for _ in range(2)]
    pa.pa_cache_store(ctx, *rows, None, *cache)
    q = torch.randn(B, Hk, 1, D, generator=g).to(torch.bfloat16).cuda()
    out = [torch.empty_like(q), torch.empty(B, Hk, 1, device="cuda")]
    want = [x.clone() for x in out]
    size = pa.cache_attn_workspace(ctx, q, cache[0]).numel()
    pa.pa_cache_attn(ctx, q, *cache, None, *want)
    big = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    current, stream = (torch.cuda.Stream(), other) if handle == "side" else (other, 0)
    with torch.cuda.stream(current):
        for _ in range(3):
            held = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
            for _ in range(4):                                  # keeps the current stream busy
                big2 = big @ big
            copy = held.clone()
            del held, big2                                      # free for the current stream's next work
            pa.pa_cache_attn(ctx, q, *cache, None, *out, stream=stream)
            torch.cuda.synchronize()
            assert bool((copy == 7).all())
            assert all(torch.equal(a, b) for a, b in zip(want, out))
    ctx.sync_status()
    ctx.close()
