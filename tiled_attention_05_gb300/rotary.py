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
    """Strides (batch, head, token) of a [B, H, T, d] operand, checked."""
    if x.dim() != 4:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected [{B}, H, {T}, {d}]")
    xB, _, xT, xd = x.shape
    if xB != B or xT != T or xd != d:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected [{B}, H, {T}, {d}]")
    if not x.is_cuda or x.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a CUDA {torch.bfloat16} tensor")
    if x.get_device() != device.index:
        raise ValueError(f"{name} is on {x.device}, expected {device} (all tensors on one GPU)")
    sb, sh, st, sd = x.stride()
    if (sd != 1 or (sb | sh | st) & 7 or x.data_ptr() & 15) and x.numel():
        raise ValueError(f"{name} needs contiguous channels, strides of a multiple of 8 elements and 16-byte alignment")
    return sb, sh, st


def _rows_positions(positions, axes, B, T, device):
    """positions (or a copy with contiguous tokens), and its strides over axes
    and batch rows (0 over what is shared)."""
    p = positions
    if p.dtype != torch.int32 and p.dtype != torch.int64:
        raise ValueError("positions must be int32 or int64")
    shape = tuple(p.shape)
    full = shape if len(shape) == 3 else (1,) + shape if len(shape) == 2 and axes == 1 else \
        (axes, 1, shape[1]) if len(shape) == 2 and shape[0] == axes else (1, 1) + shape if axes == 1 else shape
    if len(full) != 3 or full[0] != axes or full[1] not in (1, B) or full[2] != T:
        raise ValueError(f"positions has shape {shape}, expected [{axes}, {B}, {T}] or [{axes}, {T}]")
    if not p.is_cuda or p.get_device() != device.index:
        raise ValueError(f"positions is on {p.device}, expected {device} (all tensors on one GPU)")
    if T > 1 and p.stride(-1) != 1:
        p = p.contiguous()
    st = p.stride()
    if len(shape) == 3:
        return p, st[0], st[1] if full[1] == B else 0
    if len(shape) == 2:
        return (p, 0, st[0] if full[1] == B else 0) if axes == 1 else (p, st[0], 0)
    return p, 0, 0


def _call(Q, K, positions, inv_freq, sections, interleaved, inverse, Qo, Ko, stream, where):
    if Q.dim() != 4:
        raise ValueError("Q, K must be [B, H, T, d]")
    B, Hq, T, d = Q.shape
    half = inv_freq.numel()
    if inv_freq.dim() != 1 or 2 * half > d:
        raise ValueError(f"inv_freq has shape {tuple(inv_freq.shape)}, expected [rot / 2] with rot <= {d}")
    sections = (half,) if sections is None else tuple(sections)
    axes = len(sections)
    if not 1 <= axes <= 4 or min(sections) < 0 or sum(sections) != half:
        raise ValueError(f"sections {list(sections)}: one to four axes whose frequencies add up to {half}")
    device = Q.device
    q_strides = _heads(Q, "Q", B, T, d, device)
    k_strides = _heads(K, "K", B, T, d, device)
    if inv_freq.dtype != torch.float32 or inv_freq.get_device() != device.index or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be a contiguous CUDA {torch.float32} tensor on {device}")
    Hk, bf = K.shape[1], torch.bfloat16
    if Qo is not None:
        _fa._check_all(device, [(Qo, "Qo", Q.shape, bf)])
    if Ko is not None:
        _fa._check_all(device, [(Ko, "Ko", K.shape, bf)])
    handle, given = _fa._stream_ptr(stream, device), (Qo, Ko)
    lib = _fa.load()
    with _fa._under(stream, device):  # (copied positions belong to the stream that reads them)
        pos, pos_axis, pos_batch = _rows_positions(positions, axes, B, T, device)
        if Qo is None:
            Qo = torch.empty((B, Hq, T, d), dtype=bf, device=device)
        if Ko is None:
            Ko = torch.empty((B, Hk, T, d), dtype=bf, device=device)
        dims = _fa.FaRotaryDims(B, Hq, Hk, T, d, 2 * half, axes, 1 if interleaved else 0, pos.element_size(), sections,
                                q_strides, k_strides, (Hq * T * d, T * d, d), (Hk * T * d, T * d, d), pos_axis, pos_batch)
        code = lib.fa_rotary(ctypes.byref(dims), Q.data_ptr(), K.data_ptr(), pos.data_ptr(), inv_freq.data_ptr(),
                             Qo.data_ptr(), Ko.data_ptr(), inverse, handle)
    if stream is not None:
        _fa._hand_over(device, (Qo, Ko), given)
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
    """Saves the positions and frequencies only.  Its gradient is the rotation back,
    which is differentiated in turn where a graph of the gradient is asked for."""

    @staticmethod
    def forward(ctx, Q, K, positions, inv_freq, sections, interleaved, inverse=0):
        turn = fa_rotary_backward if inverse else fa_rotary
        Qr, Kr = turn(Q, K, positions, inv_freq, sections, interleaved)
        ctx.save_for_backward(positions, inv_freq)
        ctx.sections, ctx.interleaved, ctx.inverse = sections, interleaved, inverse
        return Qr, Kr

    @staticmethod
    def backward(ctx, dQr, dKr):
        positions, inv_freq = ctx.saved_tensors
        dQr, dKr = _dense(dQr), _dense(dKr)
        if torch.is_grad_enabled():
            dQ, dK = _Rotary.apply(dQr, dKr, positions, inv_freq, ctx.sections, ctx.interleaved, 1 - ctx.inverse)
        else:
            turn = fa_rotary if ctx.inverse else fa_rotary_backward
            dQ, dK = turn(dQr, dKr, positions, inv_freq, ctx.sections, ctx.interleaved)
        return dQ, dK, None, None, None, None, None


def _dense(g):
    """A gradient as the kernel takes it (an expanded or channel-strided one is copied)."""
    ok = g.stride(3) == 1 and all(s % 8 == 0 for s in g.stride()[:3]) and g.data_ptr() % 16 == 0
    return g if ok else g.contiguous()


def rotary(Q, K, positions, inv_freq, sections=None, interleaved=False):
    if inv_freq.requires_grad:
        raise ValueError("inv_freq has no gradient here; detach it")
    return _Rotary.apply(Q, K, positions, inv_freq, None if sections is None else tuple(sections), interleaved)
