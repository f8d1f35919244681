"""Python binding of the GB300 tiled exact attention library (include/fa.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libfa_gb300.so``.  There is no CPU or PyTorch fallback -- if the
library cannot be loaded, every entry point raises.

Entry points mirror the C ABI:
    fa_forward(Q, K, V, causal, scale=None, window=0)            -> (O, L)
    fa_backward(Q, K, V, O, dO, L, causal, scale=None, window=0)  -> (dQ, dK, dV)
        both also with softcap=, slopes= (score modifications) and mask= (a plan)
    fa_mask_plan(B, Tq, Tk, causal, doc_q, doc_k, prefix)         -> MaskPlan
    fa_backward_workspace_bytes(...), fa_backward_workspace_min_bytes(...), fa_status_string(code),
    fa_last_device_status()
    fa_rotary(Q, K, positions, inv_freq, ...)                     -> (Qr, Kr)
    fa_rotary_backward(dQr, dKr, positions, inv_freq, ...)        -> (dQ, dK)
    fa_cache_write(cache, K, V, tables, starts, counts=None)      (a KVCache: pages in bf16 or e4m3)
    fa_cache_read(cache, tables, lengths, T)                      -> (K, V)
    fa_cache_attention(Q, cache, tables, lengths, ...)            -> (O, L)
plus ``FlashAttention`` (a torch.autograd.Function that keeps only Q, K, V, O
and L for the backward pass) and ``attention`` (its functional form), and
``rotary`` (multi-axis rotary positions of Q and K, differentiable).

Tensors are CUDA bf16, contiguous, [B, H, T, d]; L is fp32 [B, Hq, Tq].  The
rotary calls also take strided Q and K (views of a packed projection).

Calls run on the current stream, or on ``stream=``.  Inputs have to be ready there,
and the caller orders its use of the results; what the call allocates belongs to
that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from . import build as _build

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)

EXPORTED_SYMBOLS = ("fa_forward", "fa_backward", "fa_backward_stages", "fa_backward_workspace_bytes",
                    "fa_backward_workspace_min_bytes", "fa_backward_noalloc", "fa_status_string",
                    "fa_last_device_status", "fa_last_launch_count", "fa_rotary", "fa_mask_plan_bytes", "fa_mask_plan",
                    "fa_forward_scored", "fa_backward_scored", "fa_forward_scored_workspace_bytes",
                    "fa_backward_scored_workspace_bytes", "fa_cache_write", "fa_cache_read", "fa_cache_attention",
                    "fa_cache_attention_workspace_bytes")
FA_ERR_SCRATCH_TOO_SMALL, FA_ERR_BAD_TABLE = 5, 6
FA_NOALLOC_SCRATCH_BYTES = 32 << 20
FA_BWD_PRE, FA_BWD_MAIN, FA_BWD_CAST, FA_BWD_ALL = 1, 2, 4, 7


class FAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (status {code})")


class FaDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("Tq", ctypes.c_int),
                ("Tk", ctypes.c_int), ("d", ctypes.c_int), ("dv", ctypes.c_int), ("causal", ctypes.c_int),
                ("scale", ctypes.c_float), ("window", ctypes.c_int)]


class FaScores(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("plan", ctypes.c_void_p)]


class FaRotaryDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "Hq", "Hk", "T", "d", "rot", "axes", "interleaved", "pos_bytes")] + \
        [("section", ctypes.c_int * 4)] + \
        [(n, ctypes.c_longlong * 3) for n in ("q_stride", "k_stride", "qo_stride", "ko_stride")] + \
        [("pos_axis_stride", ctypes.c_longlong), ("pos_batch_stride", ctypes.c_longlong)]


class FaCacheDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "Hq", "Hkv", "T", "d", "dv", "pages", "page", "table_pages", "quantised")]


class FaKVCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("K", "V", "k_scale", "v_scale")]


class FaCacheScores(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p),
                ("window", ctypes.c_int)]


class FaCachePrefix(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int), ("table_pages", ctypes.c_int), ("tables", ctypes.c_void_p),
                ("lengths", ctypes.c_void_p), ("starts", ctypes.c_void_p)]


_HERE = contextlib.nullcontext()
_lock = threading.Lock()
_lib = None


def lib_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Load (building first if needed) the shared library; raises if that fails."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or _build.build()
            if not os.path.exists(p):
                raise RuntimeError(f"CUDA attention library missing: {p}")
            lib = ctypes.CDLL(p)
            vp, dp = ctypes.c_void_p, ctypes.POINTER(FaDims)
            lib.fa_forward.argtypes = [dp, vp, vp, vp, vp, vp, vp]
            lib.fa_forward.restype = ctypes.c_int
            lib.fa_backward.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
            lib.fa_backward.restype = ctypes.c_int
            lib.fa_backward_stages.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t,
                                               ctypes.c_int, vp]
            lib.fa_backward_stages.restype = ctypes.c_int
            lib.fa_backward_noalloc.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
            lib.fa_backward_noalloc.restype = ctypes.c_int
            lib.fa_backward_workspace_bytes.argtypes = [dp]
            lib.fa_backward_workspace_bytes.restype = ctypes.c_size_t
            lib.fa_backward_workspace_min_bytes.argtypes = [dp]
            lib.fa_backward_workspace_min_bytes.restype = ctypes.c_size_t
            lib.fa_status_string.argtypes = [ctypes.c_int]
            lib.fa_status_string.restype = ctypes.c_char_p
            lib.fa_last_device_status.argtypes = [vp]
            lib.fa_last_device_status.restype = ctypes.c_int
            lib.fa_last_launch_count.argtypes = []
            lib.fa_last_launch_count.restype = ctypes.c_int
            sp = ctypes.POINTER(FaScores)
            lib.fa_mask_plan_bytes.argtypes = [dp]
            lib.fa_mask_plan_bytes.restype = ctypes.c_size_t
            lib.fa_mask_plan.argtypes = [dp, vp, vp, vp, ctypes.c_int, vp, ctypes.c_size_t, vp]
            lib.fa_mask_plan.restype = ctypes.c_int
            lib.fa_backward_scored_workspace_bytes.argtypes = [dp, sp]
            lib.fa_backward_scored_workspace_bytes.restype = ctypes.c_size_t
            lib.fa_forward_scored_workspace_bytes.argtypes = [dp, sp]
            lib.fa_forward_scored_workspace_bytes.restype = ctypes.c_size_t
            lib.fa_forward_scored.argtypes = [dp, sp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
            lib.fa_forward_scored.restype = ctypes.c_int
            lib.fa_backward_scored.argtypes = [dp, sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t,
                                               ctypes.c_int, vp]
            lib.fa_backward_scored.restype = ctypes.c_int
            lib.fa_rotary.argtypes = [ctypes.POINTER(FaRotaryDims), vp, vp, vp, vp, vp, vp, ctypes.c_int, vp]
            lib.fa_rotary.restype = ctypes.c_int
            cd, cc, cp = ctypes.POINTER(FaCacheDims), ctypes.POINTER(FaKVCache), ctypes.POINTER(FaCachePrefix)
            strides = ctypes.POINTER(ctypes.c_longlong)
            lib.fa_cache_write.argtypes = [cd, cc, vp, vp, strides, strides, vp, vp, vp, vp]
            lib.fa_cache_write.restype = ctypes.c_int
            lib.fa_cache_read.argtypes = [cd, cc, vp, vp, vp, vp, vp]
            lib.fa_cache_read.restype = ctypes.c_int
            lib.fa_cache_attention_workspace_bytes.argtypes = [cd, cp]
            lib.fa_cache_attention_workspace_bytes.restype = ctypes.c_size_t
            lib.fa_cache_attention.argtypes = [cd, cc, ctypes.POINTER(FaCacheScores), cp, vp, vp, vp, vp, vp, vp,
                                               ctypes.c_size_t, vp]
            lib.fa_cache_attention.restype = ctypes.c_int
            _lib = lib
    return _lib


def status_string(code: int) -> str:
    return load().fa_status_string(int(code)).decode()


fa_status_string = status_string


def make_dims(B, Hq, Hkv, Tq, Tk, d, dv, causal, scale, window: int = 0) -> FaDims:
    return FaDims(int(B), int(Hq), int(Hkv), int(Tq), int(Tk), int(d), int(dv), int(bool(causal)),
                  float(scale) if scale is not None else 0.0, int(window))


def _dims_of(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, causal, scale, window: int = 0) -> FaDims:
    if Q.dim() != 4 or K.dim() != 4 or V.dim() != 4:
        raise ValueError("Q, K, V must be [B, H, T, d]")
    B, Hq, Tq, d = Q.shape
    Bk, Hkv, Tk, dk = K.shape
    Bv, Hv, Tv, dv = V.shape
    if not (B == Bk == Bv and Hkv == Hv and Tk == Tv and d == dk):
        raise ValueError(f"inconsistent shapes Q{tuple(Q.shape)} K{tuple(K.shape)} V{tuple(V.shape)}")
    return make_dims(B, Hq, Hkv, Tq, Tk, d, dv, causal, scale, window)


def _check(t: torch.Tensor, name: str, dtype=torch.bfloat16):
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


def _check_all(device, specs):
    """The library sees only pointers, so every size it relies on is checked
    here: each (tensor, name, shape, dtype) must have exactly that shape, be a
    contiguous CUDA tensor of that dtype and live on ``device``.  Shapes are
    checked first so a mismatch is reported as such on any device."""
    index = device.index if device.type == "cuda" else -2
    for t, _, shape, dtype in specs:  # (a call's host time is mostly such checks: first without words)
        if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
            break
    else:
        return
    for t, name, shape, _ in specs:
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    for t, name, _, dtype in specs:
        _check(t, name, dtype)
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device} (all tensors on one GPU)")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the current stream's handle, without an object


def _stream_ptr(stream=None, device=None) -> int:
    if stream is None:
        if device is not None and _raw_stream is not None:
            return _raw_stream(device.index)
        stream = torch.cuda.current_stream(device)
    if device is not None and stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
    return stream.cuda_stream


def _current_device() -> int:
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else torch.cuda.current_device()


def _on(device):
    """Makes ``device`` current for a call (nothing to do where it already is)."""
    return _HERE if device.index == _current_device() else torch.cuda.device(device)


def _under(stream, device):
    """Makes ``device`` and the stream of a call current (nothing to do for the
    current one): what the call allocates and copies is then ordered with its
    kernels.  (A block from another stream's pool may still be in use there.)"""
    return _on(device) if stream is None else torch.cuda.stream(stream)


def _hand_over(device, results, given=()):
    """Results that a call made (were not given to it) under an explicit stream go to
    the caller, whose current stream may still use them when they are freed."""
    here = torch.cuda.current_stream(device)
    for n, t in enumerate(results):
        if n >= len(given) or given[n] is None:
            t.record_stream(here)


def _raise(code: int, where: str):
    if code != FA_OK:
        raise FAError(code, where)


def fa_backward_workspace_bytes(dims: FaDims) -> int:
    """Workspace for the backward's fastest schedule (what fa_backward allocates)."""
    return int(load().fa_backward_workspace_bytes(ctypes.byref(dims)))


def fa_backward_workspace_min_bytes(dims: FaDims) -> int:
    """The least workspace fa_backward accepts (then no work item is split)."""
    return int(load().fa_backward_workspace_min_bytes(ctypes.byref(dims)))


class MaskPlan:
    """Which keys each row sees, for one batch of sequences (see fa_mask_plan)."""

    def __init__(self, key, buffer):
        self.key, self.buffer = key, buffer  # (B, Tq, Tk, causal, window), int32 device array


def fa_mask_plan(B, Tq, Tk, causal: bool, window: int = 0, doc_q=None, doc_k=None, prefix=None, stream=None) -> MaskPlan:
    """The mask plan of a batch of sequences, for ``mask=`` of fa_forward,
    fa_backward and attention; built on the GPU by one small kernel.

    doc_q [B, Tq], doc_k [B, Tk]: int32 document ids; a row sees the keys of its
    own document.  Negative ids are padding.  prefix: int32 [B] or [B, Tq]; a row
    also sees the first ``prefix`` keys (causal, without a window).  The plan is
    valid for any heads, head sizes and scores with the same B, Tq, Tk, causal
    and window, as long as the ids it was built from hold."""
    dims = make_dims(B, 1, 1, Tq, Tk, 64, 64, causal, None, window)
    if (doc_q is None) != (doc_k is None):
        raise ValueError("doc_q and doc_k go together")
    if doc_q is None and prefix is None:
        raise ValueError("a mask plan needs documents or a prefix")
    if prefix is not None and prefix.dim() not in (1, 2):
        raise ValueError(f"prefix has shape {tuple(prefix.shape)}, expected ({B},) or ({B}, {Tq})")
    specs = [] if doc_q is None else [(doc_q, "doc_q", (B, Tq), torch.int32), (doc_k, "doc_k", (B, Tk), torch.int32)]
    if prefix is not None:
        specs.append((prefix, "prefix", (B,) if prefix.dim() == 1 else (B, Tq), torch.int32))
    device = specs[0][0].device
    _check_all(device, specs)
    lib = load()
    nbytes = int(lib.fa_mask_plan_bytes(ctypes.byref(dims)))
    handle = _stream_ptr(stream, device)
    with _under(stream, device):
        buffer = torch.empty(max(nbytes // 4, 4), dtype=torch.int32, device=device)
        code = lib.fa_mask_plan(ctypes.byref(dims), _ptr(doc_q), _ptr(doc_k), _ptr(prefix),
                                int(prefix is not None and prefix.dim() == 2), buffer.data_ptr(), nbytes, handle)
    if stream is not None:
        _hand_over(device, (buffer,))
    _raise(code, "fa_mask_plan")
    return MaskPlan(_plan_key(dims), buffer)


def _plan_key(dims: FaDims):
    return (dims.B, dims.Tq, dims.Tk, dims.causal, dims.window)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _scores(dims: FaDims, device, softcap, slopes, mask, stream):
    """The fa_scores of a call (None for an unmodified one), checked."""
    if slopes is None and mask is None and not softcap:
        return None
    if slopes is not None:
        if slopes.requires_grad:
            raise ValueError("slopes have no gradient here; detach them")
        _check_all(device, [(slopes, "slopes", (dims.Hq,), torch.float32)])
    if mask is not None:
        if not isinstance(mask, MaskPlan):
            raise ValueError("mask must be a MaskPlan (see fa_mask_plan)")
        if mask.key != _plan_key(dims):
            raise ValueError(f"mask was planned for (B, Tq, Tk, causal, window) = {mask.key}, the call has "
                             f"{_plan_key(dims)}")
        if mask.buffer.device != device:
            raise ValueError(f"mask is on {mask.buffer.device}, expected {device} (all tensors on one GPU)")
        if stream is not None:
            mask.buffer.record_stream(stream)
    return FaScores(float(softcap or 0.0), _ptr(slopes), None if mask is None else mask.buffer.data_ptr())


def fa_forward(Q, K, V, causal: bool, scale: float | None = None, O=None, L=None, stream=None, window: int = 0,
               softcap: float = 0.0, slopes=None, mask: MaskPlan | None = None):
    """O, L = attention forward.  Optional preallocated O / L are written in place.
    ``window=W`` (causal only) lets each row see at most its last W keys.

    ``softcap=c`` replaces each scaled score x by c tanh(x / c); ``slopes`` (fp32
    [Hq]) then subtracts slopes[h] |i + Tk - Tq - j|; ``mask`` (a MaskPlan of the
    same sizes, causal and window) hides other documents' keys and shows a
    prefix.  The backward takes the same three.  With a cap, values of V are to
    be below 2^20 in magnitude."""
    dims = _dims_of(Q, K, V, causal, scale, window)
    bf, f32 = torch.bfloat16, torch.float32
    specs = [(Q, "Q", Q.shape, bf), (K, "K", K.shape, bf), (V, "V", V.shape, bf)]
    if O is not None:
        specs.append((O, "O", (dims.B, dims.Hq, dims.Tq, dims.dv), bf))
    if L is not None:
        specs.append((L, "L", (dims.B, dims.Hq, dims.Tq), f32))
    _check_all(Q.device, specs)
    device = Q.device
    lib, ref = load(), ctypes.byref(dims)
    scores = _scores(dims, device, softcap, slopes, mask, stream)
    handle, given = _stream_ptr(stream, device), (O, L)
    with _under(stream, device):
        if O is None:
            O = torch.empty_like(Q) if dims.dv == dims.d else torch.empty(dims.B, dims.Hq, dims.Tq, dims.dv, dtype=bf,
                                                                          device=device)
        if L is None:
            L = torch.empty((dims.B, dims.Hq, dims.Tq), dtype=f32, device=device)
        nbytes = lib.fa_forward_scored_workspace_bytes(ref, scores) if scores is not None else 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
        code = lib.fa_forward_scored(ref, scores, Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
                                     L.data_ptr(), _ptr(workspace), nbytes, handle)
    if stream is not None:
        _hand_over(device, (O, L), given)
    _raise(code, "fa_forward")
    return O, L


def fa_backward(Q, K, V, O, dO, L, causal: bool, scale: float | None = None, dQ=None, dK=None, dV=None,
                workspace=None, stream=None, stages: int = FA_BWD_ALL, window: int = 0, softcap: float = 0.0,
                slopes=None, mask: MaskPlan | None = None):
    """dQ, dK, dV = attention backward from the saved O and L (``softcap``,
    ``slopes`` and ``mask`` as in the forward).

    ``stages`` selects which of the three backward kernels to launch (see
    fa_backward_stages in include/fa.h); the default runs all of them.
    """
    dims, handle, dQ, dK, dV = _backward_operands(Q, K, V, O, dO, L, causal, scale, window, dQ, dK, dV, stream)
    lib, device, ref = load(), Q.device, ctypes.byref(dims)
    scores = _scores(dims, device, softcap, slopes, mask, stream)
    with _under(stream, device):
        if workspace is None:
            need = lib.fa_backward_scored_workspace_bytes(ref, scores)
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
        elif not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous CUDA tensor on {device}")
        nbytes = workspace.numel() * workspace.element_size()
        code = lib.fa_backward_scored(ref, scores, Q.data_ptr(), K.data_ptr(), V.data_ptr(),
                                      O.data_ptr(), dO.data_ptr(), L.data_ptr(), dQ.data_ptr(), dK.data_ptr(),
                                      dV.data_ptr(), workspace.data_ptr(), nbytes, int(stages), handle)
    _raise(code, "fa_backward")
    return dQ, dK, dV


def _backward_operands(Q, K, V, O, dO, L, causal, scale, window, dQ, dK, dV, stream):
    """Dims and stream of a backward call, its gradient buffers (allocated when not
    given) and the shape / dtype / device checks of all eleven tensors."""
    dims = _dims_of(Q, K, V, causal, scale, window)
    bf, f32 = torch.bfloat16, torch.float32
    qv, rows = (dims.B, dims.Hq, dims.Tq, dims.dv), (dims.B, dims.Hq, dims.Tq)
    specs = [(Q, "Q", Q.shape, bf), (K, "K", K.shape, bf), (V, "V", V.shape, bf),
             (O, "O", qv, bf), (dO, "dO", qv, bf), (L, "L", rows, f32)]
    specs += [(t, n, like.shape, bf) for t, n, like in ((dQ, "dQ", Q), (dK, "dK", K), (dV, "dV", V))
              if t is not None]
    _check_all(Q.device, specs)
    handle, given = _stream_ptr(stream, Q.device), (dQ, dK, dV)
    with _under(stream, Q.device):
        dQ = torch.empty_like(Q) if dQ is None else dQ
        dK = torch.empty_like(K) if dK is None else dK
        dV = torch.empty_like(V) if dV is None else dV
    if stream is not None:
        _hand_over(Q.device, (dQ, dK, dV), given)
    return dims, handle, dQ, dK, dV


def fa_backward_noalloc(Q, K, V, O, dO, L, causal: bool, scale: float | None = None, dQ=None, dK=None, dV=None,
                        stream=None, window: int = 0):
    """fa_backward without a workspace, for callers that cannot allocate device
    memory: the library's fixed scratch array (FA_NOALLOC_SCRATCH_BYTES per
    GPU) is used instead.  Pass preallocated dQ / dK / dV to allocate nothing
    at all; calls that could overlap on the GPU must be ordered by the caller."""
    dims, handle, dQ, dK, dV = _backward_operands(Q, K, V, O, dO, L, causal, scale, window, dQ, dK, dV, stream)
    lib = load()
    with torch.cuda.device(Q.device):
        code = lib.fa_backward_noalloc(ctypes.byref(dims), Q.data_ptr(), K.data_ptr(), V.data_ptr(),
                                       O.data_ptr(), dO.data_ptr(), L.data_ptr(), dQ.data_ptr(), dK.data_ptr(),
                                       dV.data_ptr(), handle)
    _raise(code, "fa_backward_noalloc")
    return dQ, dK, dV


def fa_last_device_status(stream=None) -> int:
    return int(load().fa_last_device_status(_stream_ptr(stream)))


def last_launch_count() -> int:
    return int(load().fa_last_launch_count())


class _LastGradient(torch.autograd.Function):
    """Hands gradients on as a function of what they were made of, with no derivative
    (torch's once_differentiable looks at dO alone)."""

    @staticmethod
    def forward(ctx, Q, K, V, dO, dQ, dK, dV):
        return dQ, dK, dV

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the gradient of attention cannot be differentiated again")


class FlashAttention(torch.autograd.Function):
    """Autograd wrapper: saves Q, K, V (inputs) plus O and L -- nothing quadratic
    (and with modified scores the slopes and the mask plan).  Its gradient has no
    gradient: asking for one raises."""

    @staticmethod
    def forward(ctx, Q, K, V, causal=False, scale=None, window=0, softcap=0.0, slopes=None, mask=None):
        O, L = fa_forward(Q, K, V, causal, scale, window=window, softcap=softcap, slopes=slopes, mask=mask)
        plan = None if mask is None else mask.buffer
        ctx.save_for_backward(*(t for t in (Q, K, V, O, L, slopes, plan) if t is not None))
        ctx.causal, ctx.scale, ctx.window, ctx.softcap = causal, scale, window, softcap
        ctx.has_slopes, ctx.plan_key = slopes is not None, None if mask is None else mask.key
        return O

    @staticmethod
    def backward(ctx, dO):
        Q, K, V, O, L, *more = ctx.saved_tensors
        slopes = more.pop(0) if ctx.has_slopes else None
        mask = None if ctx.plan_key is None else MaskPlan(ctx.plan_key, more[0])
        dQ, dK, dV = fa_backward(Q, K, V, O, dO.contiguous(), L, ctx.causal, ctx.scale, window=ctx.window,
                                 softcap=ctx.softcap, slopes=slopes, mask=mask)
        if torch.is_grad_enabled():  # a graph of the gradient is asked for (create_graph)
            dQ, dK, dV = _LastGradient.apply(Q, K, V, dO, dQ, dK, dV)
        return dQ, dK, dV, None, None, None, None, None, None


def attention(Q, K, V, causal=False, scale=None, window=0, softcap=0.0, slopes=None, mask=None, docs=None,
              prefix=None):
    """Differentiable attention; ``softcap``, ``slopes`` and ``mask`` as in
    fa_forward (with its limit on V under a cap).  ``docs`` (int32 ids [B, T] of rows and keys, or a pair for
    each) and ``prefix`` plan the mask here, for this call and its backward;
    a program with several layers plans once (fa_mask_plan) and passes ``mask``."""
    if docs is not None or prefix is not None:
        if mask is not None:
            raise ValueError("mask is a plan already: give docs and prefix to fa_mask_plan")
        if Q.dim() != 4 or K.dim() != 4:
            raise ValueError("Q, K, V must be [B, H, T, d]")
        doc_q, doc_k = docs if isinstance(docs, (tuple, list)) else (docs, docs)
        mask = fa_mask_plan(Q.shape[0], Q.shape[2], K.shape[2], causal, window, doc_q, doc_k, prefix)
    return FlashAttention.apply(Q, K, V, causal, scale, window, softcap, slopes, mask)


from .cache import (KVCache, fa_cache_attention, fa_cache_attention_workspace_bytes, fa_cache_read,  # noqa: E402
                    fa_cache_write)
from .rotary import fa_rotary, fa_rotary_backward, rotary  # noqa: E402
