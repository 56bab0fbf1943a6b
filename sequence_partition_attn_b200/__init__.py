"""Python binding of libpa: partition attention with attention-state merge, selective reuse
and partition importance on one B200 (sm_100a).

Argument marshalling only -- every step of the path runs in libpa's CUDA kernels.  Tensors
are passed as device pointers (``tensor.data_ptr()``), partition offsets and reuse masks as
host arrays, and the stream is the current PyTorch CUDA stream unless one is given.  The
names follow the C ABI in ``include/pa.h``:

    pa_init / Context            pa_partition_attn    pa_merge_states
    pa_importance                pa_relayout_seq2head pa_sync_status / pa_wait_status
    pa_merge_states_noalloc      pa_compose_states    pa_state_drift
    pa_attn_backward             pa_cache_store       pa_cache_attn

There is no fallback: if ``libpa.so`` is missing or the device is not sm_100 the calls
raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

import numpy as np

__all__ = [
    "PA_F32", "PA_BF16", "PAError", "Context", "lib", "lib_path",
    "pa_partition_attn", "pa_merge_states", "pa_importance", "pa_relayout_seq2head",
    "pa_merge_states_noalloc", "pa_compose_states", "pa_state_drift", "pa_selftest_wait", "EXPORTED",
    "pa_relayout_seq2head_at",
    "pa_attn_backward", "pa_cache_store", "pa_cache_attn", "cache_attn_workspace", "PA_CACHE_BLOCK",
    "select_fresh",
    "predict_fresh",
]

PA_F32, PA_BF16 = 0, 1
PA_MAX_P = 128
PA_CACHE_BLOCK = 64                     # tokens that share a scale in the 8-bit K/V cache
_ERRORS = {-1: "PA_EINVAL", -2: "PA_EALIGN", -3: "PA_EUNSUPPORTED", -4: "PA_ENOMEM",
           -5: "PA_ECUDA", -6: "PA_ETIMEOUT"}
EXPORTED = ("pa_init", "pa_destroy", "pa_last_error", "pa_sync_status", "pa_wait_status", "pa_version",
            "pa_partition_attn", "pa_merge_states", "pa_importance", "pa_relayout_seq2head",
            "pa_merge_states_noalloc", "pa_compose_states", "pa_state_drift", "pa_selftest_wait",
            "pa_relayout_seq2head_at", "pa_attn_backward", "pa_cache_store", "pa_cache_attn",
            "pa_cache_attn_ws")

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "libpa.so")


class PAError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{_ERRORS.get(code, code)}: {msg}")
        self.code = code


class _AttnDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int),
                ("N", ctypes.c_int), ("D", ctypes.c_int), ("scale", ctypes.c_float),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("P", ctypes.c_int), ("part_off", ctypes.c_void_p), ("G", ctypes.c_int),
                ("fresh", ctypes.c_void_p), ("o_part", ctypes.c_void_p),
                ("lse_part", ctypes.c_void_p)]


class _MergeDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int),
                ("N", ctypes.c_int), ("D", ctypes.c_int), ("P", ctypes.c_int),
                ("G", ctypes.c_int), ("part_off", ctypes.c_void_p),
                ("o_fresh", ctypes.c_void_p), ("lse_fresh", ctypes.c_void_p),
                ("o_cached", ctypes.c_void_p), ("lse_cached", ctypes.c_void_p),
                ("fresh", ctypes.c_void_p), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("w", ctypes.c_void_p), ("cached_per_group", ctypes.c_int)]


# The descriptors of the calls below, packed in the C compiler's layout (native alignment) into
# a bytes object: about a third of a ctypes.Structure's time, which single-token calls notice.
_ATTN_BWD = struct.Struct("@iiiiif" + "P" * 7 + "iPiP" + "P" * 4)
_CACHE_STORE = struct.Struct("@iiiiii" + "P" * 7)
_CACHE_ATTN = struct.Struct("@iiiiiiif" + "P" * 9 + "N")


_LIB = None


def lib():
    """Load libpa.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m sequence_partition_attn_b200.build`")
        L = ctypes.CDLL(path)
        vp, ci = ctypes.c_void_p, ctypes.c_int
        L.pa_init.argtypes = [ci, ctypes.POINTER(vp)]
        L.pa_destroy.argtypes = [vp]
        L.pa_destroy.restype = None
        L.pa_last_error.argtypes = [vp]
        L.pa_last_error.restype = ctypes.c_char_p
        L.pa_sync_status.argtypes = [vp, vp]
        L.pa_wait_status.argtypes = [vp, vp, ctypes.c_double]
        L.pa_version.restype = ctypes.c_char_p
        L.pa_partition_attn.argtypes = [vp, ctypes.POINTER(_AttnDesc), vp]
        L.pa_merge_states.argtypes = [vp, ctypes.POINTER(_MergeDesc), vp]
        L.pa_merge_states_noalloc.argtypes = [ctypes.POINTER(_MergeDesc), vp]
        L.pa_importance.argtypes = [vp, ci, ci, ci, ci, ci, vp, vp, vp, vp, vp]
        L.pa_compose_states.argtypes = [vp, ci, ci, ci, ci, ci, ci, ci, vp, vp, vp, vp, vp]
        L.pa_relayout_seq2head.argtypes = [vp, vp, vp, ci, ci, ci, ci, ci, ci, vp]
        L.pa_relayout_seq2head_at.argtypes = [vp, vp, vp, ci, ci, ci, ci, ci, ci, vp]
        L.pa_state_drift.argtypes = [vp, ci, ci, ci, ci, ci, ci, ci, vp, vp, vp, vp, vp, vp, vp]
        L.pa_selftest_wait.argtypes = [vp, ctypes.c_double, vp]
        L.pa_attn_backward.argtypes = [vp, vp, vp]
        L.pa_cache_store.argtypes = [vp, vp, vp]
        L.pa_cache_attn.argtypes = [vp, vp, vp]
        L.pa_cache_attn_ws.argtypes = [vp, ci, ci, ci, ci, ci, ci, ci, ctypes.POINTER(ctypes.c_size_t)]
        for f in ("pa_init", "pa_sync_status", "pa_wait_status", "pa_partition_attn", "pa_merge_states", "pa_merge_states_noalloc",
                  "pa_compose_states", "pa_state_drift", "pa_selftest_wait",
                  "pa_importance", "pa_relayout_seq2head", "pa_relayout_seq2head_at",
                  "pa_attn_backward", "pa_cache_store", "pa_cache_attn", "pa_cache_attn_ws"):
            getattr(L, f).restype = ci
        _LIB = L
    return _LIB


def _check(ctx_ptr, rc):
    if rc != 0:
        msg = lib().pa_last_error(ctx_ptr)
        raise PAError(rc, msg.decode() if msg else "")


class Context:
    """A libpa context on one device (pa_init / pa_destroy)."""

    def __init__(self, device: int = 0):
        self._ptr = ctypes.c_void_p()
        _check(None, lib().pa_init(device, ctypes.byref(self._ptr)))
        self.device = device

    @property
    def ptr(self):
        return self._ptr

    def sync_status(self, stream=None, timeout=None):
        """pa_sync_status: synchronise the stream, raise if a device wait gave up.  With
        `timeout` (seconds), pa_wait_status: raise PAError (PA_ETIMEOUT) if the stream's
        work has not finished by then (nothing is cancelled)."""
        if timeout is None:
            _check(self._ptr, lib().pa_sync_status(self._ptr, _stream(stream)))
        else:
            _check(self._ptr, lib().pa_wait_status(self._ptr, _stream(stream), float(timeout)))

    def close(self):
        if self._ptr:
            lib().pa_destroy(self._ptr)
            self._ptr = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return PA_BF16
    if t.dtype == torch.float32:
        return PA_F32
    raise PAError(-3, f"dtype {t.dtype} not supported")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _host_i32(a):
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _host_u8(a):
    return None if a is None else np.ascontiguousarray(np.asarray(a, dtype=np.uint8))


def pa_partition_attn(ctx: Context, q, k, v, part_off, G, fresh, o_part, lse_part,
                      scale=None, stream=None):
    """Per-partition attention states (O_p, LSE_p) for the fresh (query group, KV group)
    pairs.  q, k, v: [B, H, N, D] CUDA tensors (bf16 or f32); o_part [P, B, H, N, D];
    lse_part [P, B, H, N] f32; part_off int[P+1]; fresh uint8 [QG, KG] or None."""
    B, H, N, D = q.shape
    off = _host_i32(part_off)
    fr = _host_u8(fresh)
    d = _AttnDesc(_dtype_code(q), B, H, N, D,
                  float(scale if scale is not None else 1.0 / np.sqrt(D)),
                  q.data_ptr(), k.data_ptr(), v.data_ptr(), len(off) - 1,
                  off.ctypes.data, int(G), None if fr is None else fr.ctypes.data,
                  o_part.data_ptr(), lse_part.data_ptr())
    _check(ctx.ptr, lib().pa_partition_attn(ctx.ptr, ctypes.byref(d), _stream(stream)))


def pa_merge_states(ctx: Context, part_off, G, fresh, o_fresh, lse_fresh, o_cached, lse_cached,
                    o, lse, w=None, stream=None, cached_per_group=False):
    """Merge fresh / cached states per the mask; o [B, H, N, D], lse [B, H, N]; w [QG, P]
    (fused importance) optional.  cached_per_group: the cache holds one composed state per
    KV group ([KG, B, H, N, D], from pa_compose_states)."""
    P, B, H, N, D = o_fresh.shape
    off = _host_i32(part_off)
    fr = _host_u8(fresh)
    d = _MergeDesc(_dtype_code(o_fresh), B, H, N, D, P, int(G), off.ctypes.data,
                   o_fresh.data_ptr(), lse_fresh.data_ptr(),
                   None if o_cached is None else o_cached.data_ptr(),
                   None if lse_cached is None else lse_cached.data_ptr(),
                   None if fr is None else fr.ctypes.data, o.data_ptr(), lse.data_ptr(),
                   None if w is None else w.data_ptr(), 1 if cached_per_group else 0)
    _check(ctx.ptr, lib().pa_merge_states(ctx.ptr, ctypes.byref(d), _stream(stream)))


def pa_compose_states(ctx: Context, o_part, lse_part, factor, o_group, lse_group, stream=None):
    """Compose every `factor` consecutive partitions' states into one (no recomputation):
    o_part [P, B, H, N, D], lse_part [P, B, H, N] -> o_group [C, ...], lse_group [C, ...]."""
    P, B, H, N, D = o_part.shape
    _check(ctx.ptr, lib().pa_compose_states(ctx.ptr, _dtype_code(o_part), B, H, N, D, P, int(factor),
                                            o_part.data_ptr(), lse_part.data_ptr(),
                                            o_group.data_ptr(), lse_group.data_ptr(), _stream(stream)))


def pa_merge_states_noalloc(part_off, G, fresh, o_fresh, lse_fresh, o_cached, lse_cached, o, lse,
                            w=None, stream=None):
    """pa_merge_states without a context and without any device allocation: the fused
    importance uses libpa's fixed 4 MiB scratch array (for callers that must not call
    cudaMalloc).  Calls that overlap on the GPU share that scratch and must not be issued
    concurrently."""
    P, B, H, N, D = o_fresh.shape
    off = _host_i32(part_off)
    fr = _host_u8(fresh)
    d = _MergeDesc(_dtype_code(o_fresh), B, H, N, D, P, int(G), off.ctypes.data,
                   o_fresh.data_ptr(), lse_fresh.data_ptr(),
                   None if o_cached is None else o_cached.data_ptr(),
                   None if lse_cached is None else lse_cached.data_ptr(),
                   None if fr is None else fr.ctypes.data, o.data_ptr(), lse.data_ptr(),
                   None if w is None else w.data_ptr())
    _check(None, lib().pa_merge_states_noalloc(ctypes.byref(d), _stream(stream)))


def pa_importance(ctx: Context, part_off, G, lse_part, lse, w, stream=None):
    """w[qg, p] = mean over b, h, rows of qg of exp(lse_part - lse); w [QG, P] overwritten."""
    P, B, H, N = lse_part.shape
    off = _host_i32(part_off)
    _check(ctx.ptr, lib().pa_importance(ctx.ptr, B, H, N, P, int(G), off.ctypes.data,
                                        lse_part.data_ptr(), lse.data_ptr(), w.data_ptr(),
                                        _stream(stream)))


def pa_state_drift(ctx: Context, part_off, G, sel, o_new, o_ref, d2, r2, stream=None):
    """Per (query group, partition) sums of (o_new - o_ref)^2 and o_ref^2 over the pairs
    selected by sel (uint8 [QG, KG] or None = all): o_new, o_ref [P, B, H, N, D];
    d2, r2 [QG, P] f32, overwritten (0 for unselected pairs)."""
    P, B, H, N, D = o_new.shape
    off = _host_i32(part_off)
    sl = _host_u8(sel)
    _check(ctx.ptr, lib().pa_state_drift(ctx.ptr, _dtype_code(o_new), B, H, N, D, P, int(G),
                                         off.ctypes.data, None if sl is None else sl.ctypes.data,
                                         o_new.data_ptr(), o_ref.data_ptr(), d2.data_ptr(),
                                         r2.data_ptr(), _stream(stream)))


def pa_selftest_wait(ctx: Context, seconds=0.05, stream=None):
    """Launch the bounded-wait self-test: a wait that nothing completes gives up after
    `seconds`; the next ctx.sync_status() raises PAError with code PA_ETIMEOUT."""
    _check(ctx.ptr, lib().pa_selftest_wait(ctx.ptr, float(seconds), _stream(stream)))


def pa_relayout_seq2head(ctx: Context, src, dst, n_chunks=1, chunk=-1, stream=None):
    """dst[h, n, :] = src[n, h, :] for sequence chunk `chunk` of `n_chunks` (-1 = all)."""
    N, H, D = src.shape
    _check(ctx.ptr, lib().pa_relayout_seq2head(ctx.ptr, src.data_ptr(), dst.data_ptr(), N, H, D,
                                               src.element_size(), int(n_chunks), int(chunk),
                                               _stream(stream)))


def pa_relayout_seq2head_at(ctx: Context, src, dst, tok0, stream=None):
    """dst[h, tok0 + n, :] = src[n, h, :]: src [n_tok, H, D] placed at token tok0 of
    dst [H, N, D] (one piece of a chunked sequence-parallel all-to-all)."""
    n_tok, H, D = src.shape
    _check(ctx.ptr, lib().pa_relayout_seq2head_at(ctx.ptr, src.data_ptr(), dst.data_ptr(), n_tok, H, D,
                                                  src.element_size(), dst.shape[-2], int(tok0),
                                                  _stream(stream)))


def _want(ctx, name, t, shape, dtype):
    """Check a tensor argument: the kernels take raw pointers to contiguous device memory."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != ctx.device or not t.is_contiguous():
        _refuse(ctx, name, t, shape, dtype)
    return t.data_ptr()


def _refuse(ctx, name, t, shape, dtype):
    if t.shape != shape:
        raise PAError(-1, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise PAError(-3, f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.get_device() != ctx.device:
        raise PAError(-1, f"{name} is on {t.device}, the context on cuda:{ctx.device}")
    raise PAError(-1, f"{name} is not contiguous")


def _maybe(ctx, name, t, shape, dtype):
    return 0 if t is None else _want(ctx, name, t, shape, dtype)


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _code(t):
    """pa_dtype of a tensor."""
    code = _CODES.get(t.dtype)
    if code is None:
        code = _CODES[t.dtype] = _dtype_code(t)
    return code


_CODES = {}


def _call(ctx, rc):
    if rc != 0:
        _check(ctx._ptr, rc)


def _four(name, t):
    if t.dim() != 4:
        raise PAError(-1, f"{name} has shape {tuple(t.shape)}, expected four dimensions")
    return t.shape


def _scale(scale, D):
    return float(scale) if scale is not None else D ** -0.5


def _address(a):
    return 0 if a is None else a.__array_interface__["data"][0]


def _raw_stream(ctx, stream):
    if stream is None:
        return _torch()._C._cuda_getCurrentRawStream(ctx.device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _allocating_for(ctx, stream):
    """Torch allocates for the stream of this handle.  Memory comes from what was freed for the same
    stream, whose work may still use it, and goes back there: right for work on that stream only."""
    torch = _torch()
    if stream == torch._C._cuda_getCurrentRawStream(ctx.device):
        return contextlib.nullcontext()
    # 0 is the default stream; as an external handle torch would take it for "none given"
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=ctx.device) if stream
                             else torch.cuda.default_stream(ctx.device))


def pa_attn_backward(ctx: Context, q, k, v, o, lse, do, part_off, G, fresh, dq, dk, dv, delta,
                     dlse=None, scale=None, stream=None):
    """Gradients dq, dk, dv (overwritten, [B, H, N, D]) of the fresh pairs of a merged output
    (o [B, H, N, D], lse [B, H, N]) from the loss's gradients do and, optionally, dlse.
    Reused states are constants; a row without a fresh pair gets zeros.  delta [B, H, N] f32
    receives do.o - dlse and is the call's only scratch.  part_off, G, fresh and scale as in
    the forward call."""
    torch = _torch()
    full = B, H, N, D = _four("q", q)
    row, dt, f32 = (B, H, N), q.dtype, torch.float32
    code = _code(q)
    off, fr, G = _host_i32(part_off), _host_u8(fresh), int(G)
    _want_mask(off, G, fr)
    d = _ATTN_BWD.pack(
        code, B, H, N, D, _scale(scale, D), _want(ctx, "q", q, full, dt), _want(ctx, "k", k, full, dt),
        _want(ctx, "v", v, full, dt), _want(ctx, "o", o, full, dt), _want(ctx, "lse", lse, row, f32),
        _want(ctx, "do", do, full, dt), _maybe(ctx, "dlse", dlse, row, f32), off.size - 1, _address(off), G,
        _address(fr), _want(ctx, "dq", dq, full, dt), _want(ctx, "dk", dk, full, dt),
        _want(ctx, "dv", dv, full, dt), _want(ctx, "delta", delta, row, f32))
    _call(ctx, lib().pa_attn_backward(ctx._ptr, d, _raw_stream(ctx, stream)))


def _want_mask(off, G, fr):
    """The C call reads P + 1 offsets and ceil(P / G)^2 mask entries."""
    P = off.size - 1
    if off.ndim != 1 or P < 1 or not 1 <= G <= P:
        raise PAError(-1, f"part_off of {off.size} entries with G={G}")
    QG = -(-P // G)
    if fr is not None and fr.size != QG * QG:
        raise PAError(-1, f"fresh has {fr.size} entries, expected {QG} x {QG}")


def _cache_args(ctx, kc, vc, k_scale, v_scale):
    torch = _torch()
    full = B, Hk, M, D = _four("kc", kc)
    code = torch.uint8 if kc.dtype is torch.uint8 else torch.float8_e4m3fn
    blocks = (B, Hk, -(-M // PA_CACHE_BLOCK))
    return (B, Hk, M, D, _want(ctx, "kc", kc, full, code), _want(ctx, "vc", vc, full, code),
            _want(ctx, "k_scale", k_scale, blocks, torch.float32),
            _want(ctx, "v_scale", v_scale, blocks, torch.float32))


def pa_cache_store(ctx: Context, k, v, start, kc, vc, k_scale, v_scale, stream=None):
    """Round k, v [B, Hk, T, D] (bf16 or f32) into the 8-bit cache kc, vc [B, Hk, M, D]
    (float8_e4m3fn, or uint8 holding the codes) with scales [B, Hk, ceil(M / 64)] f32, at token
    offsets start (int32 [B] on the device, or None for 0)."""
    torch = _torch()
    B, Hk, M, D, pk, pv, pks, pvs = _cache_args(ctx, kc, vc, k_scale, v_scale)
    T = _four("k", k)[2]
    rows = (B, Hk, T, D)
    d = _CACHE_STORE.pack(_code(k), B, Hk, T, M, D, _want(ctx, "k", k, rows, k.dtype),
                          _want(ctx, "v", v, rows, k.dtype), _maybe(ctx, "start", start, (B,), torch.int32),
                          pk, pv, pks, pvs)
    _call(ctx, lib().pa_cache_store(ctx._ptr, d, _raw_stream(ctx, stream)))


def cache_attn_workspace(ctx: Context, q, kc):
    """Scratch for pa_cache_attn on tensors of these shapes (uint8, maybe empty).  Calls that
    may overlap on the GPU, and captured graphs that may, need one each."""
    import torch
    B, H, Nq, D = _four("q", q)
    n = ctypes.c_size_t()
    _check(ctx.ptr, lib().pa_cache_attn_ws(ctx.ptr, _dtype_code(q), B, H, kc.shape[1], Nq, kc.shape[2], D,
                                           ctypes.byref(n)))
    return torch.empty(n.value, dtype=torch.uint8, device=torch.device("cuda", ctx.device))


def pa_cache_attn(ctx: Context, q, kc, vc, k_scale, v_scale, lens, o, lse, scale=None, workspace=None,
                  stream=None):
    """Attention state (o [B, H, Nq, D], lse [B, H, Nq] f32) of q against the first lens[b]
    tokens (int32 [B] on the device, or None for all M) of the 8-bit cache; H is a multiple of
    the cache's Hk.  No causal mask: all Nq rows of a request see the same tokens.
    workspace: from cache_attn_workspace; without one the call takes it from
    torch's allocator, for the stream it runs on."""
    torch = _torch()
    B, Hk, M, D, pk, pv, pks, pvs = _cache_args(ctx, kc, vc, k_scale, v_scale)
    _, H, Nq, _ = _four("q", q)
    rows, dt = (B, H, Nq, D), q.dtype
    pq = _want(ctx, "q", q, rows, dt)
    s = _raw_stream(ctx, stream)
    if workspace is None:
        with _allocating_for(ctx, s):
            workspace = cache_attn_workspace(ctx, q, kc)
    size = workspace.numel()
    d = _CACHE_ATTN.pack(_code(q), B, H, Hk, Nq, M, D, _scale(scale, D), pq, pk, pv, pks, pvs,
                         _maybe(ctx, "lens", lens, (B,), torch.int32), _want(ctx, "o", o, rows, dt),
                         _want(ctx, "lse", lse, (B, H, Nq), torch.float32),
                         _want(ctx, "workspace", workspace, (size,), torch.uint8) if size else 0, size)
    _call(ctx, lib().pa_cache_attn(ctx._ptr, d, s))


def select_fresh(w_stored, G: int, threshold: float) -> np.ndarray:
    """Host reuse selection from stored importance: uint8[QG, KG], 1 where some partition of
    the KV group has stored importance at or above the threshold (recompute), else 0
    (reuse the cached states).  DiTango web summary, Methodology 1 (anchor-guided
    selection, group-wise decisions)."""
    w = np.asarray(w_stored, dtype=np.float64)
    QG, P = w.shape
    KG = -(-P // G)
    pad = np.full((QG, KG * G), -np.inf)
    pad[:, :P] = w
    return (pad.reshape(QG, KG, G).max(axis=2) >= threshold).astype(np.uint8)


def predict_fresh(w_stored, d2, r2, G: int, eps: float) -> np.ndarray:
    """Host reuse selection between anchors from predicted error (DiTango web summary,
    Methodology 1, "Error modelling" and "Online Prediction"): the error of reusing the
    states of partition p for query group qg grows with its stored importance times the
    drift of the states; the drift of the remote states is estimated by that of the own
    KV group's states, which are recomputed every step:
        drift[qg] = sqrt(sum_{p in own group} d2[qg, p] / sum_{p in own group} r2[qg, p]).
    Returns uint8[QG, KG]: 1 (recompute) where max_{p in kg} w_stored[qg, p] * drift[qg]
    reaches eps, and always on the diagonal (own group); d2, r2 as from pa_state_drift."""
    w = np.asarray(w_stored, dtype=np.float64)
    d2 = np.asarray(d2, dtype=np.float64)
    r2 = np.asarray(r2, dtype=np.float64)
    QG, P = w.shape
    KG = -(-P // G)
    own = (np.arange(P)[None, :] // G) == np.arange(QG)[:, None]
    num = np.where(own, d2, 0.0).sum(axis=1)
    den = np.where(own, r2, 0.0).sum(axis=1)
    drift = np.sqrt(np.divide(num, den, out=np.zeros_like(num), where=den > 0))
    pad = np.full((QG, KG * G), -np.inf)
    pad[:, :P] = w * drift[:, None]
    m = (pad.reshape(QG, KG, G).max(axis=2) >= eps).astype(np.uint8)
    m[np.arange(QG), np.arange(QG)] = 1
    return m
