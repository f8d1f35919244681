"""Rotary positions of Q and K with one to four position axes (fa_rotary in
include/fa.h): argument checks and marshalling, and the differentiable form.

    fa_rotary(Q, K, positions, inv_freq, sections=None, interleaved=False)            -> (Qr, Kr)
    fa_rotary_backward(dQr, dKr, positions, inv_freq, sections=None, interleaved=False) -> (dQ, dK)
    rotary(Q, K, positions, inv_freq, sections=None, interleaved=False)               -> (Qr, Kr), differentiable

Q [B, Hq, T, d] and K [B, Hk, T, d] are CUDA bf16 with contiguous channels; the
other strides are free (multiples of 8 elements), so views of a packed
projection [B, T, heads * d] are taken as they are.  Results are contiguous
[B, H, T, d], as the attention takes them.

positions (int32 or int64) is [axes, B, T], or [axes, T] for all batch rows; with
one axis also [B, T] or [T].  inv_freq is fp32 [rot / 2] with rot <= d: the
channels past rot are copied.  sections gives each axis its number of frequencies
(default: one axis with all of them).
"""
from __future__ import annotations

import ctypes

import torch

import tiled_attention_05_gb300 as _fa


def _heads(x, name, B, T, d, device):
    if x.dim() != 4 or x.shape[0] != B or x.shape[2] != T or x.shape[3] != d:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected [{B}, H, {T}, {d}]")
    if not x.is_cuda or x.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a CUDA {torch.bfloat16} tensor")
    if x.device != device:
        raise ValueError(f"{name} is on {x.device}, expected {device} (all tensors on one GPU)")
    if x.numel() and (x.stride(3) != 1 or any(s % 8 for s in x.stride()[:3]) or x.data_ptr() % 16):
        raise ValueError(f"{name} needs contiguous channels, strides of a multiple of 8 elements and 16-byte alignment")


def _rows_positions(positions, axes, B, T, device):
    """positions as a view [axes, B, T] (stride 0 over what is shared)."""
    p = positions
    if p.dtype not in (torch.int32, torch.int64):
        raise ValueError("positions must be int32 or int64")
    if p.dim() == 1 and axes == 1:
        p = p.view(1, 1, -1)
    elif p.dim() == 2:
        p = p.unsqueeze(0) if axes == 1 else p.unsqueeze(1)
    if p.dim() != 3 or p.shape[0] != axes or p.shape[1] not in (1, B) or p.shape[2] != T:
        raise ValueError(f"positions has shape {tuple(positions.shape)}, expected [{axes}, {B}, {T}] or [{axes}, {T}]")
    if not p.is_cuda or p.device != device:
        raise ValueError(f"positions is on {p.device}, expected {device} (all tensors on one GPU)")
    p = p.expand(axes, B, T)
    return p if T <= 1 or p.stride(2) == 1 else p.contiguous()


def _call(Q, K, positions, inv_freq, sections, interleaved, inverse, Qo, Ko, stream, where):
    if Q.dim() != 4:
        raise ValueError("Q, K must be [B, H, T, d]")
    B, Hq, T, d = Q.shape
    if inv_freq.dim() != 1 or 2 * inv_freq.numel() > d:
        raise ValueError(f"inv_freq has shape {tuple(inv_freq.shape)}, expected [rot / 2] with rot <= {d}")
    rot = 2 * inv_freq.numel()
    sections = [rot // 2] if sections is None else [int(n) for n in sections]
    if not 1 <= len(sections) <= 4 or min(sections) < 0 or 2 * sum(sections) != rot:
        raise ValueError(f"sections {sections}: one to four axes whose frequencies add up to {rot // 2}")
    _heads(Q, "Q", B, T, d, Q.device)
    _heads(K, "K", B, T, d, Q.device)
    if not inv_freq.is_cuda or inv_freq.dtype != torch.float32 or not inv_freq.is_contiguous() or \
            inv_freq.device != Q.device:
        raise ValueError(f"inv_freq must be a contiguous CUDA {torch.float32} tensor on {Q.device}")
    pos = _rows_positions(positions, len(sections), B, T, Q.device)
    if pos is not positions and stream is not None:
        pos.record_stream(stream)
    outs = []
    for x, o, name in ((Q, Qo, "Qo"), (K, Ko, "Ko")):
        if o is None:
            o = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            _fa._check_all(Q.device, [(o, name, x.shape, torch.bfloat16)])
        outs.append(o)
    (Qo, Ko), Hk = outs, K.shape[1]
    c = ctypes.c_int * 4
    s3 = ctypes.c_longlong * 3
    dims = _fa.FaRotaryDims(B, Hq, Hk, T, d, rot, len(sections), int(bool(interleaved)), pos.element_size(),
                            c(*sections), s3(*Q.stride()[:3]), s3(*K.stride()[:3]), s3(*Qo.stride()[:3]),
                            s3(*Ko.stride()[:3]), pos.stride(0), pos.stride(1))
    lib = _fa.load()
    with torch.cuda.device(Q.device):
        code = lib.fa_rotary(ctypes.byref(dims), Q.data_ptr(), K.data_ptr(), pos.data_ptr(), inv_freq.data_ptr(),
                             Qo.data_ptr(), Ko.data_ptr(), inverse, _fa._stream_ptr(stream, Q.device))
    _fa._raise(code, where)
    return Qo, Ko


def fa_rotary(Q, K, positions, inv_freq, sections=None, interleaved=False, Qo=None, Ko=None, stream=None):
    """Qr, Kr = Q and K turned by their positions.  Qo / Ko: preallocated
    contiguous results (Q and K themselves where those are contiguous)."""
    return _call(Q, K, positions, inv_freq, sections, interleaved, 0, Qo, Ko, stream, "fa_rotary")


def fa_rotary_backward(dQr, dKr, positions, inv_freq, sections=None, interleaved=False, dQ=None, dK=None, stream=None):
    """dQ, dK from the gradients of fa_rotary's results: the rotation back."""
    return _call(dQr, dKr, positions, inv_freq, sections, interleaved, 1, dQ, dK, stream, "fa_rotary_backward")


class _Rotary(torch.autograd.Function):
    """Saves the positions and frequencies only."""

    @staticmethod
    def forward(ctx, Q, K, positions, inv_freq, sections, interleaved):
        Qr, Kr = fa_rotary(Q, K, positions, inv_freq, sections, interleaved)
        ctx.save_for_backward(positions, inv_freq)
        ctx.sections, ctx.interleaved = sections, interleaved
        return Qr, Kr

    @staticmethod
    def backward(ctx, dQr, dKr):
        positions, inv_freq = ctx.saved_tensors
        dQ, dK = fa_rotary_backward(_dense(dQr), _dense(dKr), positions, inv_freq, ctx.sections, ctx.interleaved)
        return dQ, dK, None, None, None, None


def _dense(g):
    """A gradient as the kernel takes it (an expanded or channel-strided one is copied)."""
    ok = g.stride(3) == 1 and all(s % 8 == 0 for s in g.stride()[:3]) and g.data_ptr() % 16 == 0
    return g if ok else g.contiguous()


def rotary(Q, K, positions, inv_freq, sections=None, interleaved=False):
    if inv_freq.requires_grad:
        raise ValueError("inv_freq has no gradient here; detach it")
    return _Rotary.apply(Q, K, positions, inv_freq, None if sections is None else tuple(sections), interleaved)
