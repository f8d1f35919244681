"""The paged key/value cache and attention over it (fa_cache_* in include/fa.h):
argument checks and marshalling.

    KVCache(K, V, k_scale=None, v_scale=None), KVCache.empty(pages, Hkv, page, d, ...)
    fa_cache_write(cache, K, V, tables, starts, counts=None)
    fa_cache_read(cache, tables, lengths, T)                               -> (K, V)
    fa_cache_attention(Q, cache, tables, lengths, ..., prefix=None)        -> (O, L)
    fa_cache_attention_workspace_bytes(Q, cache, tables, prefix=None)

A program keeps a pool of pages (KVCache) for each layer, and for all of them the
tables: int32 [B, n], the pages of each sequence in their order.  After the rotary
step the new tokens' K and V are written behind what is cached, and their Q
attends over it:

    fa_cache_write(cache, K, V, tables, lengths)           # K, V [B, Hkv, T, d]: T new tokens each
    O, L = fa_cache_attention(Q, cache, tables, lengths + T)

Tables, lengths, starts and counts stay on the GPU and are not looked at by the host;
an index in them that does not fit reaches no memory, and fa_last_device_status
reports FA_ERR_BAD_TABLE.  The calls have no gradient.
"""
from __future__ import annotations

import ctypes

import torch

import tiled_attention_05_gb300 as _fa

PAGE_SIZES = (16, 32, 64, 128, 256)


class KVCache:
    """Pools of pages: K [pages, Hkv, page, d] and V [pages, Hkv, page, dv], both bf16 or both
    float8_e4m3fn, the latter with fp32 scales [pages, Hkv, page].  Holds the tensors it is
    given and copies nothing; another tensor is another cache."""

    def __init__(self, K, V, k_scale=None, v_scale=None):
        if K.dim() != 4 or V.dim() != 4 or K.shape[:3] != V.shape[:3]:
            raise ValueError(f"K and V must be [pages, Hkv, page, d] and [pages, Hkv, page, dv], got {tuple(K.shape)} and "
                             f"{tuple(V.shape)}")
        if K.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError("a cache is bfloat16 or float8_e4m3fn")
        self.quantised = K.dtype == torch.float8_e4m3fn
        if (k_scale is None) != (not self.quantised) or (v_scale is None) != (not self.quantised):
            raise ValueError("float8_e4m3fn caches have k_scale and v_scale, bfloat16 caches have none")
        pages, Hkv, page, _ = K.shape
        if page not in PAGE_SIZES:
            raise ValueError(f"a page has {PAGE_SIZES} positions, not {page}")
        specs = [(K, "K", K.shape, K.dtype), (V, "V", V.shape, K.dtype)]
        if self.quantised:
            specs += [(k_scale, "k_scale", (pages, Hkv, page), torch.float32),
                      (v_scale, "v_scale", (pages, Hkv, page), torch.float32)]
        self.device = K.device
        _fa._check_all(self.device, specs)
        self.K, self.V, self.k_scale, self.v_scale = K, V, k_scale, v_scale
        self._sizes = {}  # dims and workspace of the attention calls by their sizes
        self._shape, self._dv = tuple(K.shape), V.shape[3]
        self._where = [f for t in (K, V, k_scale, v_scale) if t is not None for f in (t.data_ptr, t.numel)]
        self._at = [f() for f in self._where]
        self._pools = ctypes.byref(_fa.FaKVCache(K.data_ptr(), V.data_ptr(), _fa._ptr(k_scale), _fa._ptr(v_scale)))

    def _struct(self):
        """The library's fa_kv_cache.  Refused if a tensor was given other memory since."""
        if [f() for f in self._where] != self._at:
            raise ValueError("a pool of the cache has moved since; make another KVCache of it")
        return self._pools

    def __setattr__(self, name, value):
        if name in ("K", "V", "k_scale", "v_scale") and "_pools" in self.__dict__:
            raise AttributeError(f"a KVCache keeps the {name} that it was made of")
        object.__setattr__(self, name, value)

    @classmethod
    def empty(cls, pages, Hkv, page, d, dv=None, dtype=torch.bfloat16, device="cuda"):
        """A new cache of zeros."""
        quantised = dtype == torch.float8_e4m3fn
        K, V = (torch.zeros(pages, Hkv, page, w, dtype=torch.uint8 if quantised else dtype, device=device)
                for w in (d, d if dv is None else dv))
        if not quantised:
            return cls(K, V)
        scales = (torch.zeros(pages, Hkv, page, device=device) for _ in range(2))
        return cls(K.view(dtype), V.view(dtype), *scales)

    def _dims(self, B, Hq, T, table_pages):
        pages, Hkv, page, d = self._shape
        return _fa.FaCacheDims(B, Hq, Hkv, T, d, self._dv, pages, page, table_pages, self.quantised)


def _table(t, name, rows):
    """Columns of a table of ``rows`` rows (None: any), as far as its shape goes."""
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [{'sequences' if rows is None else rows}, pages]")
    return t.shape[1]


def _new_rows(x, name, shape, device):
    """Strides (batch, head, token) of a [B, Hkv, T, w] operand, checked."""
    if tuple(x.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected {shape}")
    if not x.is_cuda or x.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a CUDA {torch.bfloat16} tensor")
    if x.get_device() != device.index:
        raise ValueError(f"{name} is on {x.device}, expected {device} (all tensors on one GPU)")
    sb, sh, st, sd = x.stride()
    if x.numel() and (sd != 1 or (sb | sh | st) & 7 or x.data_ptr() & 15):
        raise ValueError(f"{name} needs contiguous channels, strides of a multiple of 8 elements and 16-byte alignment")
    return (ctypes.c_longlong * 3)(*((sb, sh, st) if x.numel() else (0, 0, 0)))


def fa_cache_write(cache: KVCache, K, V, tables, starts, counts=None, stream=None):
    """Writes tokens K [B, Hkv, T, d] and V [B, Hkv, T, dv] (bf16; views as fa_rotary takes
    them) to positions starts[b] .. starts[b] + T - 1 of each sequence, quantised if the
    cache is; with counts [B] only the first counts[b] tokens of each."""
    if K.dim() != 4:
        raise ValueError("K, V must be [B, Hkv, T, d]")
    B, _, T, _ = K.shape
    _, Hkv, _, d = cache._shape
    device = cache.device
    ks = _new_rows(K, "K", (B, Hkv, T, d), device)
    vs = _new_rows(V, "V", (B, Hkv, T, cache._dv), device)
    n, i32 = _table(tables, "tables", B), torch.int32
    specs = [(tables, "tables", tables.shape, i32), (starts, "starts", (B,), i32)]
    if counts is not None:
        specs.append((counts, "counts", (B,), i32))
    _fa._check_all(device, specs)
    dims, handle = cache._dims(B, 0, T, n), _fa._stream_ptr(stream, device)
    with _fa._under(stream, device):
        code = _fa.load().fa_cache_write(ctypes.byref(dims), cache._struct(), K.data_ptr(), V.data_ptr(), ks, vs,
                                         tables.data_ptr(), starts.data_ptr(), _fa._ptr(counts), handle)
    _fa._raise(code, "fa_cache_write")


def fa_cache_read(cache: KVCache, tables, lengths, T: int, K=None, V=None, stream=None):
    """K [B, Hkv, T, d], V [B, Hkv, T, dv] (bf16) = positions 0 .. T - 1 of each sequence, zero
    from lengths[b] on.  Optional preallocated K / V are written in place."""
    device = cache.device
    n, B = _table(tables, "tables", None), tables.shape[0]
    _, Hkv, _, d = cache._shape
    T, dv, bf, given = int(T), cache._dv, torch.bfloat16, (K, V)
    if T < 0:
        raise ValueError(f"T is {T}")
    specs = [(tables, "tables", tables.shape, torch.int32), (lengths, "lengths", (B,), torch.int32)]
    specs += [(t, name, (B, Hkv, T, w), bf) for t, name, w in ((K, "K", d), (V, "V", dv)) if t is not None]
    _fa._check_all(device, specs)
    dims, handle = cache._dims(B, 0, T, n), _fa._stream_ptr(stream, device)
    with _fa._under(stream, device):
        if K is None:
            K = torch.empty((B, Hkv, T, d), dtype=bf, device=device)
        if V is None:
            V = torch.empty((B, Hkv, T, dv), dtype=bf, device=device)
        code = _fa.load().fa_cache_read(ctypes.byref(dims), cache._struct(), tables.data_ptr(), lengths.data_ptr(),
                                        K.data_ptr(), V.data_ptr(), handle)
    if stream is not None:
        _fa._hand_over(device, (K, V), given)
    _fa._raise(code, "fa_cache_read")
    return K, V


def _attention_dims(Q, cache, tables, prefix, specs):
    """Dims, workspace bytes and fa_cache_prefix (None without one) of a call; the index
    arrays go to specs."""
    if Q.dim() != 4:
        raise ValueError("Q must be [B, Hq, T, d]")
    B, Hq, T, d = Q.shape
    if d != cache._shape[3]:
        raise ValueError(f"Q has shape {tuple(Q.shape)}, the cache's keys have {cache._shape[3]} channels")
    cols, i32, pre, groups, n = _table(tables, "tables", B), torch.int32, None, 0, 0
    specs.append((tables, "tables", tables.shape, i32))
    if prefix is not None:
        p_tables, lengths, starts = prefix if len(prefix) == 3 else (*prefix, None)
        n, groups = _table(p_tables, "prefix tables", None), p_tables.shape[0]
        specs += [(p_tables, "prefix tables", p_tables.shape, i32), (lengths, "prefix lengths", (groups,), i32)]
        if starts is not None:
            specs.append((starts, "prefix starts", (groups + 1,), i32))
        elif groups != 1:
            raise ValueError(f"{groups} prefixes need starts [{groups + 1}], the first sequence of each group")
        pre = _fa.FaCachePrefix(groups, n, p_tables.data_ptr(), lengths.data_ptr(), _fa._ptr(starts))
    key = (B, Hq, T, cols, groups, n)
    sizes = cache._sizes.get(key)
    if sizes is None:
        ref = ctypes.byref(cache._dims(B, Hq, T, cols))
        with _fa._on(cache.device):  # (it asks for the SMs)
            nbytes = int(_fa.load().fa_cache_attention_workspace_bytes(ref, pre))
        if len(cache._sizes) > 1000:
            cache._sizes.clear()
        sizes = cache._sizes[key] = (ref, nbytes)
    return (*sizes, pre)


def fa_cache_attention_workspace_bytes(Q, cache: KVCache, tables, prefix=None) -> int:
    """The workspace that fa_cache_attention needs (what it allocates without one); 0 where
    the tables hold few positions."""
    specs = []
    nbytes = _attention_dims(Q, cache, tables, prefix, specs)[1]
    _fa._check_all(cache.device, specs)
    return nbytes


def fa_cache_attention(Q, cache: KVCache, tables, lengths, scale: float | None = None, window: int = 0,
                       softcap: float = 0.0, slopes=None, prefix=None, O=None, L=None, workspace=None, stream=None):
    """O [B, Hq, T, dv], L [B, Hq, T] = attention of the last T tokens of each sequence, Q
    [B, Hq, T, d], over the lengths[b] positions that the cache holds of it (theirs among
    them): row t sees positions up to lengths[b] - T + t, and nothing where that is
    negative (O = 0, L = -inf).  ``scale``, ``window``, ``softcap`` and ``slopes`` as in
    fa_forward.

    ``prefix=(tables [S, n], lengths [S], starts [S + 1])``: sequences starts[s] ..
    starts[s + 1] - 1 share the lengths[s] positions of tables[s] in front of their own;
    their keys are read once for all of them.  Without starts one prefix serves the
    whole batch.  Pages that the window hides from all rows may be gone from the tables."""
    device, bf, f32 = cache.device, torch.bfloat16, torch.float32
    specs = [(Q, "Q", Q.shape, bf)]
    ref, nbytes, pre = _attention_dims(Q, cache, tables, prefix, specs)
    (B, Hq, T, d), dv = Q.shape, cache._dv
    specs.append((lengths, "lengths", (B,), torch.int32))
    if O is not None:
        specs.append((O, "O", (B, Hq, T, dv), bf))
    if L is not None:
        specs.append((L, "L", (B, Hq, T), f32))
    if slopes is not None:
        if slopes.requires_grad:
            raise ValueError("slopes have no gradient here; detach them")
        specs.append((slopes, "slopes", (Hq,), f32))
    _fa._check_all(device, specs)
    lib, given = _fa.load(), (O, L)
    window = max(-1, min(int(window), 2 ** 31 - 1))  # (ctypes would cut it to 32 bits)
    scores = _fa.FaCacheScores(float(scale or 0.0), float(softcap or 0.0), _fa._ptr(slopes), window)
    handle = _fa._stream_ptr(stream, device)
    with _fa._under(stream, device):
        if O is None:
            O = torch.empty_like(Q) if dv == d else torch.empty((B, Hq, T, dv), dtype=bf, device=device)
        if L is None:
            L = torch.empty((B, Hq, T), dtype=f32, device=device)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
        elif not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous CUDA tensor on {device}")
        code = lib.fa_cache_attention(ref, cache._struct(), ctypes.byref(scores), pre, Q.data_ptr(), tables.data_ptr(),
                                      lengths.data_ptr(), O.data_ptr(), L.data_ptr(), _fa._ptr(workspace),
                                      0 if workspace is None else workspace.nbytes, handle)
    if stream is not None:
        _fa._hand_over(device, (O, L), given)
    _fa._raise(code, "fa_cache_attention")
    return O, L
