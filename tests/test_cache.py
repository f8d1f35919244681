"""The key/value cache and attention over it against their definition in float64, and
the refusals of bad arguments.

Tolerances of the attention, with A = sum of p |v|, the size of what a row of O is
averaged from:
  scores  a dot product of d terms in fp32, each addition off by a last place at most:
          d 2^-23 of sum |q k| scale; a cap adds 2^-20 of itself, a bias and the
          following products 2^-21 of their sizes, and exp2, log2 and the sum 2^-19
  L       off by as much as the worst score
  O       a weight is off by twice that (itself and the sum), and by its rounding: half a
          step of bf16 (2^-8) or fp16 (2^-11, e4m3 caches); n sums in fp32, n 2^-23; all
          of A; and the result's own rounding, 2^-8 of O.
Codes and scales of written rows follow from three fp32 operations that are the same
here, and have to be equal; a row read back is one product rounded once, equal too."""
import ctypes
import math

import pytest
import torch

import tiled_attention_05_gb300 as fa

bf, f8 = torch.bfloat16, torch.float8_e4m3fn


# ---------------------------------------------------------------- refusals (CPU)
def zeros(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("args, why", [
    ((zeros(4, 2, 16), zeros(4, 2, 16, 64)), "pages, Hkv, page, d"),
    ((zeros(4, 2, 16, 64), zeros(4, 3, 16, 64)), "pages, Hkv, page, d"),
    ((zeros(4, 2, 16, 64, dtype=torch.float16),) * 2, "bfloat16 or float8_e4m3fn"),
    ((zeros(4, 2, 16, 64), zeros(4, 2, 16, 64), zeros(4, 2, 16), zeros(4, 2, 16)), "have none"),
    ((zeros(4, 2, 16, 64, dtype=torch.uint8).view(f8),) * 2, "k_scale and v_scale"),
    ((zeros(4, 2, 24, 64),) * 2, "a page has"),
    ((zeros(4, 2, 16, 64),) * 2, "CUDA"),
])
def test_cache_refuses(args, why):
    with pytest.raises(ValueError, match=why):
        fa.KVCache(*args)


def dims(**kw):
    z = dict(B=2, Hq=4, Hkv=2, T=3, d=64, dv=64, pages=8, page=16, table_pages=4, quantised=0)
    z.update(kw)
    return fa.FaCacheDims(*(z[n] for n, _ in fa.FaCacheDims._fields_))


POOLS = (0x1000, 0x2000, 0x3000, 0x4000)


def abi_write(z, pools=POOLS, k=0x5000, v=0x6000, ks=(64, 64, 64), vs=(64, 64, 64), tables=0x7000, starts=0x8000, counts=0):
    s3 = ctypes.c_longlong * 3
    return fa.load().fa_cache_write(ctypes.byref(z), ctypes.byref(fa.FaKVCache(*pools)), k, v, s3(*ks), s3(*vs), tables, starts,
                                    counts, None)


def abi_read(z, pools=POOLS, tables=0x7000, lengths=0x8000, k=0x5000, v=0x6000):
    return fa.load().fa_cache_read(ctypes.byref(z), ctypes.byref(fa.FaKVCache(*pools)), tables, lengths, k, v, None)


def abi_attention(z, pools=POOLS, scores=None, prefix=None, q=0x5000, tables=0x7000, lengths=0x8000, o=0x9000, l=0xa000,
                  ws=0x100000, nbytes=1 << 40):
    return fa.load().fa_cache_attention(ctypes.byref(z), ctypes.byref(fa.FaKVCache(*pools)), scores, prefix, q, tables, lengths, o,
                                        l, ws, nbytes, None)


BAD = [dict(B=-1), dict(T=-1), dict(Hkv=-1), dict(pages=-1), dict(page=0), dict(table_pages=-1), dict(quantised=2), dict(d=0)]
NOT_SERVED = [dict(d=96), dict(dv=32), dict(page=48), dict(page=8), dict(page=512), dict(table_pages=(1 << 26) + 1),
              dict(B=1 << 20, Hkv=1 << 12)]


@pytest.mark.parametrize("call", [abi_write, abi_read, abi_attention])
def test_abi_refuses_dims(call):
    for bad in BAD:
        assert call(dims(**bad)) == fa.FA_ERR_INVALID_ARG, bad
    for bad in NOT_SERVED:
        assert call(dims(**bad)) == fa.FA_ERR_UNSUPPORTED, bad
    for bad in ((0, 0x2000, 0, 0), (0x1008, 0x2000, 0, 0), (0x1000, 0x2001, 0, 0)):
        assert call(dims(), pools=bad) == fa.FA_ERR_INVALID_ARG
    for bad in ((0x1000, 0x2000, 0, 0x4000), (0x1000, 0x2000, 0x3000, 0x4002)):
        assert call(dims(quantised=1), pools=bad) == fa.FA_ERR_INVALID_ARG
    assert call(dims(), tables=0) == fa.FA_ERR_INVALID_ARG
    assert call(dims(), tables=0x7002) == fa.FA_ERR_INVALID_ARG
    assert call(dims(T=0)) == fa.FA_OK
    assert call(dims(B=0)) == fa.FA_OK


def test_abi_write_refuses_the_rest():
    for bad in (dict(k=0), dict(v=0x6008), dict(ks=(64, 60, 64)), dict(vs=(64, 64, 4)), dict(starts=0), dict(starts=0x8002),
                dict(counts=0x8002)):
        assert abi_write(dims(), **bad) == fa.FA_ERR_INVALID_ARG, bad


def test_abi_read_refuses_the_rest():
    for bad in (dict(k=0), dict(v=0x6008), dict(lengths=0), dict(lengths=0x8002)):
        assert abi_read(dims(), **bad) == fa.FA_ERR_INVALID_ARG, bad


def test_abi_attention_refuses_the_rest():
    S, P = fa.FaCacheScores, fa.FaCachePrefix
    for bad in (dict(ws=0), dict(ws=0x100010), dict(nbytes=0)):
        assert abi_attention(dims(table_pages=100), **bad) == fa.FA_ERR_INVALID_ARG, bad
    for bad in (dict(q=0), dict(q=0x5008), dict(o=0), dict(o=0x9008), dict(l=0xa002), dict(lengths=0), dict(scores=S(math.nan, 0, None, 0)), dict(scores=S(math.inf, 0, None, 0)),
                dict(scores=S(0, -1.0, None, 0)), dict(scores=S(0, 2000.0, None, 0)), dict(scores=S(0, math.nan, None, 0)),
                dict(scores=S(0, 0, 0x10002, 0)), dict(scores=S(0, 0, None, -1)), dict(prefix=P(-1, 4, 0x7000, 0x8000, None)),
                dict(prefix=P(1, -4, 0x7000, 0x8000, None)), dict(prefix=P(1, 4, None, 0x8000, None)),
                dict(prefix=P(1, 4, 0x7000, None, None)), dict(prefix=P(2, 4, 0x7000, 0x8000, None)),
                dict(prefix=P(1, 4, 0x7002, 0x8000, None)), dict(prefix=P(1, 4, 0x7000, 0x8000, 0x8001))):
        assert abi_attention(dims(), **bad) == fa.FA_ERR_INVALID_ARG, bad
    assert abi_attention(dims(Hq=3)) == fa.FA_ERR_INVALID_ARG
    assert abi_attention(dims(Hkv=0)) == fa.FA_ERR_INVALID_ARG
    assert abi_attention(dims(B=1 << 15, T=1 << 15)) == fa.FA_ERR_UNSUPPORTED
    assert abi_attention(dims(), prefix=P(1, (1 << 26) + 1, 0x7000, 0x8000, None)) == fa.FA_ERR_UNSUPPORTED
    # distances past 2^24 are not exact in fp32
    far = dims(table_pages=(1 << 20) + 1)
    assert abi_attention(far, scores=S(0, 0, 0x10000, 0)) == fa.FA_ERR_UNSUPPORTED
    # few positions: no workspace is asked for
    assert fa.load().fa_cache_attention_workspace_bytes(ctypes.byref(dims()), None) == 0
    z = dims(table_pages=100)
    need = fa.load().fa_cache_attention_workspace_bytes(ctypes.byref(z), None)
    assert need > 0 and abi_attention(z, nbytes=need - 1) == fa.FA_ERR_INVALID_ARG
    assert fa.load().fa_cache_attention_workspace_bytes(ctypes.byref(dims(Hq=3)), None) == 0


# ---------------------------------------------------------------- inputs
class Setup:
    """A cache with pages in no order and its sequences; what lies behind a sequence's end is
    NaN.  lens, prefix: lists; starts: the groups' (prefix given)."""

    def __init__(self, lens, Hkv, d, dv, quant, page, prefix=(), starts=None, seed=0, std=1.0, spare=2, extra_cols=1):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.lens, self.page, self.quant, self.d, self.dv, self.Hkv = lens, page, quant, d, dv, Hkv
        cols = [max(1, -(-max(max(ls, default=0), 0) // page)) + extra_cols for ls in (lens, list(prefix))]
        n = len(lens) * cols[0] + len(prefix) * cols[1] + spare
        ids = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        self.tables = ids[:len(lens) * cols[0]].view(len(lens), cols[0]).contiguous()
        self.p_tables = ids[len(lens) * cols[0]:][:len(prefix) * cols[1]].view(len(prefix), cols[1]).contiguous()
        self.lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.prefix = None
        self.p_lens, self.starts = list(prefix), starts
        if prefix:
            self.prefix = (self.p_tables, torch.tensor(prefix, dtype=torch.int32, device="cuda"))
            if starts is not None:
                self.prefix += (torch.tensor(starts, dtype=torch.int32, device="cuda"),)
        size = torch.exp(torch.randn(n, Hkv, page, 1, generator=g, device="cuda"))
        pools, scales = [], []
        for w in (d, dv):
            x = (torch.randn(n, Hkv, page, w, generator=g, device="cuda") * std * size.clamp(0.2, 5)).to(bf)
            if quant:
                codes, scale = quantise(x)
                pools.append(codes)
                scales.append(scale)
            else:
                pools.append(x)
        # rows that no position within the lengths holds
        held = torch.zeros(n, page, dtype=torch.bool, device="cuda")
        for table, ls in ((self.tables, lens), (self.p_tables, list(prefix))):
            for row, length in zip(table, ls):
                p = torch.arange(max(length, 0), device="cuda")
                held[row.long()[p // page], p % page] = True
        stale = ~held[:, None].expand(n, Hkv, page)
        for x in pools:
            raw = x.view(torch.uint8 if quant else torch.int16)
            raw[stale] = 0x7f if quant else 0x7fc0
        for x in scales:
            x[stale] = math.nan
        self.cache = fa.KVCache(*pools, *scales)

    def rows(self, table, length):
        """fp64 K, V [Hkv, length, w] of one table."""
        p = torch.arange(max(length, 0), device="cuda")
        at, off = table.long()[p // self.page], p % self.page
        out = []
        for x, s in ((self.cache.K, self.cache.k_scale), (self.cache.V, self.cache.v_scale)):
            y = x.view(torch.uint8 if self.quant else torch.int16)[at, :, off].view(x.dtype).double()
            out.append((y if s is None else y * s[at, :, off].double()[..., None]).transpose(0, 1))
        return out

    def group(self, b):
        if not self.p_lens:
            return None
        starts = self.starts or [0, len(self.lens)]
        return next((s for s in range(len(self.p_lens)) if starts[s] <= b < starts[s + 1]), None)


def quantise(x):
    a = x.float().abs().amax(-1, keepdim=True).clamp_min(2.0 ** -60)
    f = torch.full_like(a, 448.0) / a  # one rounding (448.0 / a is the product with a reciprocal: two)
    return (x.float() * f).to(f8), (a * (1.0 / 448.0)).squeeze(-1).contiguous()


def check(s, Q, O, L, scale=None, window=0, softcap=0.0, slopes=None):
    B, Hq, T, d = Q.shape
    G, scale = Hq // s.Hkv, scale or d ** -0.5
    assert torch.isfinite(O).all()
    for b, n in enumerate(s.lens):
        K, V = s.rows(s.tables[b], n)
        P, group = 0, s.group(b)
        if group is not None:
            P = max(s.p_lens[group], 0)
            pk, pv = s.rows(s.p_tables[group], P)
            K, V = torch.cat((pk, K), 1), torch.cat((pv, V), 1)
        q = Q[b].double().view(s.Hkv, G, T, d)
        x = torch.einsum("hgtd,hjd->hgtj", q, K) * scale
        size = torch.einsum("hgtd,hjd->hgtj", q.abs(), K.abs()) * scale
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        i = torch.arange(T, device="cuda").view(-1, 1) + P + n - T
        j = torch.arange(P + max(n, 0), device="cuda").view(1, -1)
        bias = torch.zeros_like(x)
        if slopes is not None:
            bias = slopes.double().view(s.Hkv, G, 1, 1) * (i - j)
        x = x - bias
        sees = ((j <= i) & (i >= P)).expand(x.shape)
        if window:
            sees = sees & (i - j < window)
        none = ~sees.any(-1)
        x = x.masked_fill(~sees, -math.inf)
        p = torch.softmax(x, -1).masked_fill(~sees, 0.0)
        Lr = torch.logsumexp(x, -1) if x.shape[-1] else torch.full(x.shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
        Or, A = torch.einsum("hgtj,hjd->hgtd", p, V), torch.einsum("hgtj,hjd->hgtd", p, V.abs())

        def top(y):
            return y.abs().masked_fill(~sees, 0.0).amax(-1) if y.shape[-1] else torch.zeros_like(Lr)

        off = d * 2.0 ** -23 * top(size) + 2.0 ** -20 * softcap + 2.0 ** -21 * (top(bias) + top(x.nan_to_num(neginf=0.0))) + 2.0 ** -19
        got_L, got_O = L[b].double().view_as(Lr), O[b].double().view_as(Or)
        assert ((got_L == -math.inf) == none).all()
        assert (got_O[none] == 0).all()
        fine = ~none
        assert ((got_L - Lr).abs()[fine] <= off[fine]).all(), float(((got_L - Lr).abs() / off)[fine].max())
        step = 2.0 ** -11 if s.quant else 2.0 ** -8
        tol = A * (step + 2 * off + x.shape[-1] * 2.0 ** -23)[..., None] + 2.0 ** -8 * Or.abs()
        bad = (got_O - Or).abs() > tol
        assert not bad.any(), (b, float(((got_O - Or).abs() / tol)[bad].max()))


def query(s, Hq, T, seed=1, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(len(s.lens), Hq, T, s.d, generator=g, device="cuda") * std).to(bf)


def slopes_of(H):
    return (2.0 ** (-8.0 * torch.arange(1, H + 1) / H)).cuda()


# ---------------------------------------------------------------- attention (GPU)
SHAPES = [
    # lens, Hq, Hkv, T, d, dv, page
    ([1], 1, 1, 1, 64, 64, 16),
    ([200], 8, 2, 1, 64, 64, 16),
    ([0, 1, 15, 16, 17, 0, 31, 32, 33, 127, 128, 129, -4], 4, 2, 1, 128, 128, 32),
    ([5000, 1, 700], 32, 8, 1, 128, 128, 64),
    ([300, 299, 2, 0, 3], 6, 2, 4, 128, 64, 16),          # rows of a short sequence that see nothing
    ([77, 1000], 16, 1, 1, 64, 128, 256),                 # 16 rows
    ([77, 1000], 34, 2, 1, 128, 128, 128),                # 17: two tiles
    ([130, 65, 40], 3, 3, 40, 64, 64, 64),                # many query rows
    ([257], 8, 2, 9, 128, 128, 16),
    ([1 + 7 * k % 61 for k in range(300)], 4, 4, 1, 64, 64, 16),  # many short sequences
    ([70001], 8, 2, 1, 128, 128, 128),                    # one long one
    ([4096] * 3, 8, 8, 2, 128, 128, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("long_tables", [False, True])  # (whole items where they hold few positions)
@pytest.mark.parametrize("lens, Hq, Hkv, T, d, dv, page", SHAPES)
def test_attention(lens, Hq, Hkv, T, d, dv, page, quant, long_tables):
    s = Setup(lens, Hkv, d, dv, quant, page, extra_cols=70 if long_tables else 1)
    Q = query(s, Hq, T, std=1.5)
    O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths)
    check(s, Q, O, L)
    again = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths)
    assert torch.equal(O, again[0]) and torch.equal(L, again[1])
    assert fa.fa_last_device_status() == fa.FA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("mods", [dict(scale=0.3), dict(softcap=5.0), dict(softcap=50.0), dict(slopes=True), dict(window=1),
                                  dict(window=100), dict(window=33, softcap=20.0, slopes=True, scale=0.2)])
@pytest.mark.parametrize("T", [1, 5])
def test_attention_modified(mods, T, quant):
    s = Setup([700, 3, 1, 0, 64, 2049], 2, 128, 128, quant, 64)
    Q, mods = query(s, 8, T, std=1.5), dict(mods)
    if mods.get("slopes"):
        mods["slopes"] = slopes_of(8)
    O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, **mods)
    check(s, Q, O, L, **mods)


PREFIXES = [
    # lens, prefix lengths, starts, Hq, Hkv, T, d, dv, page
    ([5, 0, 100], [300], None, 4, 2, 1, 128, 128, 64),
    ([40] * 7, [129], None, 8, 2, 3, 64, 64, 16),
    ([1, 2, 3, 4, 5, 6, 700, 8], [500, 0, 33, 1], [1, 3, 3, 6, 7], 8, 4, 1, 128, 64, 32),  # some without one, an empty group
    ([9, 9], [-3], None, 2, 1, 1, 64, 128, 16),
    ([20 + k for k in range(40)], [1500, 777], [0, 19, 40], 16, 2, 1, 128, 128, 128),
    ([3, 4, 0, 2], [6000], None, 12, 4, 5, 64, 64, 256),
    ([300] * 130, [257], None, 8, 1, 1, 128, 128, 64),    # 1040 rows over one prefix
    # 128 rows and fewer of a group (two parts of an item), 129 to 256, and more; one key tile and many
    ([17] * 32, [100], None, 4, 1, 1, 128, 64, 16),
    ([17, 0] * 10, [129, 5000], [0, 9, 20], 8, 2, 1, 64, 128, 32),
    ([5 + k for k in range(33)], [4000], None, 4, 1, 1, 128, 128, 256),
    ([5 + k for k in range(64)], [3001], None, 16, 4, 1, 64, 64, 64),
    ([40] * 97, [2000], None, 6, 1, 1, 64, 128, 128),
    ([9, 2, 30, 4], [20000], None, 48, 2, 3, 128, 64, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("lens, prefix, starts, Hq, Hkv, T, d, dv, page", PREFIXES)
def test_shared_prefix(lens, prefix, starts, Hq, Hkv, T, d, dv, page, quant):
    s = Setup(lens, Hkv, d, dv, quant, page, prefix, starts)
    Q = query(s, Hq, T, std=1.5)
    O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix)
    check(s, Q, O, L)
    again = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix)
    assert torch.equal(O, again[0]) and torch.equal(L, again[1])
    assert fa.fa_last_device_status() == fa.FA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("heads", [(128, 128), (64, 64)])
@pytest.mark.parametrize("mods", [dict(softcap=30.0), dict(softcap=2.0), dict(slopes=True), dict(window=40), dict(window=1),
                                  dict(window=250, softcap=20.0, slopes=True)])
def test_shared_prefix_modified(mods, quant, heads):
    s = Setup([30, 2, 0, 77, 20, 64, 3, 3], 2, *heads, quant, 32, [300, 200], [0, 5, 8])
    Q, mods = query(s, 16, 3, std=1.5), dict(mods)
    if mods.get("slopes"):
        mods["slopes"] = slopes_of(16)
    O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, **mods)
    check(s, Q, O, L, **mods)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("mods", [dict(softcap=30.0), dict(softcap=2.0), dict(slopes=True), dict(window=40), dict(window=1),
                                  dict(window=250, softcap=20.0, slopes=True)])
@pytest.mark.parametrize("T, d, dv", [(1, 128, 128), (3, 64, 64), (2, 128, 64)])
def test_shared_prefix_of_few_rows_modified(T, d, dv, mods, quant):
    s = Setup([30, 2, 0, 77, 20], 2, d, dv, quant, 64, [700, 90, 5], [0, 2, 3, 5])
    Q, mods = query(s, 8, T, std=1.5), dict(mods)
    if mods.get("slopes"):
        mods["slopes"] = slopes_of(8)
    O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, **mods)
    check(s, Q, O, L, **mods)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
def test_nan_of_a_prefix(quant):
    """A NaN key or value of a prefix reaches the rows that see it, in whatever place of a tile
    it stands, and none that a window hides it from (values in bf16 have to be finite)."""
    s = Setup([30] * 40, 1, 64, 64, quant, 16, [400, 400], [0, 20, 40])
    Q = query(s, 4, 1)
    NaN, one = (torch.full((1, 1, 1, 64), x, device="cuda").to(bf) for x in (math.nan, 1.0))
    at = torch.tensor([130], dtype=torch.int32, device="cuda")
    for K, V in ((NaN, one), (one, NaN)):
        before = [x.clone() for x in bits(s.cache)]
        fa.fa_cache_write(s.cache, K, V, s.p_tables[:1], at)
        for mods in (dict(), dict(softcap=5.0)):
            O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, **mods)
            assert torch.isnan(O[:20]).all() and torch.isfinite(O[20:]).all() and torch.isfinite(L[20:]).all()
            assert torch.isnan(L[:20]).all() == (K is NaN or quant)
            if quant or V is one:
                O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, window=250, **mods)
                assert torch.isfinite(O).all() and torch.isfinite(L).all()
        for x, y in zip(bits(s.cache), before):
            x.copy_(y)


@pytest.mark.gpu
def test_value_scales_far_apart():
    """Value rows of very different sizes, rows of zeros among them: the fp16 weights carry the scale."""
    s = Setup([900, 50], 2, 128, 128, True, 64)
    v = s.cache.v_scale
    v[::2] *= 2.0 ** 20
    v[1::2, :, ::3] *= 2.0 ** -30
    s.cache.V.view(torch.uint8)[:, :, 5] = 0
    v[:, :, 5] = 2.0 ** -60 / 448
    Q = query(s, 8, 1, std=1.5)
    check(s, Q, *fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths))


@pytest.mark.gpu
def test_query_rows_of_any_size():
    """Rows of e4m3 calls go to fp16 by a power of two of their own: 2^100 beside 2^-100."""
    s = Setup([200, 90], 1, 64, 64, True, 16)
    Q = query(s, 4, 1)
    Q[0, 1] *= 2.0 ** -100
    Q[0, 2] = 0
    s.cache.k_scale.mul_(2.0 ** -100)
    Q[1] *= 2.0 ** 100
    check(s, Q, *fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths))


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
def test_nan_reaches_the_rows_that_see_it(quant):
    s = Setup([500, 40], 2, 64, 64, quant, 16)
    K = torch.full((2, 2, 1, 64), math.nan, device="cuda").to(bf)
    V = torch.ones(2, 2, 1, 64, device="cuda").to(bf)
    at = torch.tensor([100, 39], dtype=torch.int32, device="cuda")
    fa.fa_cache_write(s.cache, K, V, s.tables, at, counts=torch.tensor([1, 1], dtype=torch.int32, device="cuda"))
    Q = query(s, 4, 3)
    O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths)
    assert torch.isnan(O[0]).all() and torch.isnan(L[0]).all()
    # the last key of sequence 1 is seen by its last row alone
    assert torch.isnan(O[1, :, 2]).all() and torch.isnan(L[1, :, 2]).all()
    assert torch.isfinite(O[1, :, :2]).all() and torch.isfinite(L[1, :, :2]).all()
    # out of the window it reaches nobody
    O, L = fa.fa_cache_attention(Q[:, :, :1].contiguous(), s.cache, s.tables, s.lengths - torch.tensor([0, 1], device="cuda").int(),
                                 window=300)
    assert torch.isfinite(O).all() and torch.isfinite(L).all()


@pytest.mark.gpu
@pytest.mark.parametrize("mods", [dict(), dict(softcap=5.0), dict(window=3)])
def test_nan_value_of_a_hidden_key(mods):
    """In e4m3 a value that a row does not see may be anything, its scale NaN too."""
    s = Setup([300, 17], 2, 64, 128, True, 16)
    K = torch.ones(2, 2, 1, 64, device="cuda").to(bf)
    V = torch.full((2, 2, 1, 128), math.nan, device="cuda").to(bf)
    fa.fa_cache_write(s.cache, K, V, s.tables, s.lengths - 1)
    Q = query(s, 4, 5)
    O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, **mods)
    assert torch.isnan(O[:, :, 4]).all() and torch.isnan(L[:, :, 4]).all()
    assert torch.isfinite(O[:, :, :4]).all() and torch.isfinite(L[:, :, :4]).all()
    # hidden by a window: from the rows after it
    more = torch.ones(2, 2, 4, 64, device="cuda").to(bf), torch.ones(2, 2, 4, 128, device="cuda").to(bf)
    fa.fa_cache_write(s.cache, *more, s.tables, s.lengths)
    O, L = fa.fa_cache_attention(Q[:, :, :2].contiguous(), s.cache, s.tables, s.lengths + 4, window=4)
    assert torch.isnan(O[:, :, 0]).all() and torch.isfinite(O[:, :, 1]).all() and torch.isfinite(L[:, :, 1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
def test_workspace_and_results_of_the_caller(quant):
    s = Setup([500, 40, 3], 2, 128, 64, quant, 16, [100], None)
    Q = query(s, 4, 2)
    need = fa.fa_cache_attention_workspace_bytes(Q, s.cache, s.tables, s.prefix)
    guard = 4096
    ws = torch.full((need + guard,), 0xff, dtype=torch.uint8, device="cuda")
    O = torch.full((3, 4, 2, 64), 7.0, device="cuda").to(bf)
    L = torch.full((3, 4, 2), 7.0, device="cuda")
    got = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, workspace=ws[:need], O=O, L=L)
    assert got[0] is O and got[1] is L
    check(s, Q, O, L)
    assert (ws[need:] == 0xff).all()
    with pytest.raises(fa.FAError):
        fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, workspace=ws[:need - 1])


@pytest.mark.gpu
def test_attention_checks_its_operands():
    s = Setup([50, 40], 2, 64, 64, False, 16)
    Q = query(s, 4, 1)
    call = lambda **kw: fa.fa_cache_attention(**{**dict(Q=Q, cache=s.cache, tables=s.tables, lengths=s.lengths), **kw})  # noqa: E731
    for bad in (dict(Q=Q[0]), dict(Q=Q[..., :32]), dict(Q=Q.float()), dict(tables=s.tables[:1]), dict(tables=s.tables.long()),
                dict(lengths=s.lengths[:1]), dict(lengths=s.lengths.cpu()), dict(slopes=torch.ones(3, device="cuda")),
                dict(prefix=(s.tables, s.lengths)), dict(prefix=(s.tables, s.lengths, s.lengths)), dict(O=Q.float()),
                dict(slopes=torch.ones(4, device="cuda", requires_grad=True)), dict(Q=Q.transpose(1, 2).contiguous().transpose(1, 2)[:, ::2])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(window=-1), dict(softcap=1e9), dict(scale=math.nan)):
        with pytest.raises(fa.FAError):
            call(**bad)
    with pytest.raises(AttributeError):
        s.cache.K = s.cache.K.clone()


# ---------------------------------------------------------------- write and read (GPU)
def write_by_torch(cache, K, V, tables, starts, counts):
    B, _, T, _ = K.shape
    page = cache.K.shape[2]
    for b in range(B):
        for t in range(min(T, counts[b])):
            p = starts[b] + t
            at, off = int(tables[b, p // page]), p % page
            for x, pool, scale in ((K, cache.K, cache.k_scale), (V, cache.V, cache.v_scale)):
                row = x[b, :, t]
                if scale is None:
                    pool[at, :, off] = row
                else:
                    codes, s = quantise(row)
                    pool.view(torch.uint8)[at, :, off] = codes.view(torch.uint8)
                    scale[at, :, off] = s


def bits(cache):
    kind = torch.uint8 if cache.quantised else torch.int16
    return [cache.K.view(kind), cache.V.view(kind)] + ([cache.k_scale, cache.v_scale] if cache.quantised else [])


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("B, Hkv, T, d, dv, page, starts, counts, packed", [
    (1, 1, 1, 64, 64, 16, [0], None, False),
    (3, 2, 5, 128, 128, 16, [0, 13, 31], [5, 0, 3], False),
    (4, 8, 1, 128, 128, 64, [63, 64, 0, 200], None, True),
    (2, 3, 67, 64, 128, 32, [1, 100], [67, 66], False),
    (2, 5, 33, 128, 64, 256, [250, 0], [33, 99], False),  # (a count past T: T tokens)
    (2, 4, 19, 64, 64, 128, [7, 120], [-2, 19], True),
])
def test_write_and_read(B, Hkv, T, d, dv, page, starts, counts, packed, quant):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    n = -(-(max(starts) + T) // page)
    cache = fa.KVCache.empty(B * n + 1, Hkv, page, d, dv, f8 if quant else bf)
    for x in bits(cache):  # what is there stays
        x.copy_(torch.randint(0, 100, x.shape, generator=g, device="cuda").to(x.dtype))
    want = fa.KVCache(*(None if x is None else x.clone() for x in (cache.K, cache.V, cache.k_scale, cache.v_scale)))
    tables = torch.randperm(B * n, generator=g, device="cuda").to(torch.int32).view(B, n)
    kv = torch.randn(B, T, 2 * Hkv, max(d, dv), generator=g, device="cuda") * torch.exp(
        3 * torch.randn(B, T, 2 * Hkv, 1, generator=g, device="cuda"))
    kv = kv.to(bf)
    kv[0, 0, 0] = 0
    K, V = kv[:, :, :Hkv, :d].transpose(1, 2), kv[:, :, Hkv:, :dv].transpose(1, 2)
    if not packed:
        K, V = K.contiguous(), V.contiguous()
    at = torch.tensor(starts, dtype=torch.int32, device="cuda")
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    fa.fa_cache_write(cache, K, V, tables, at, counts=cnt)
    write_by_torch(want, K, V, tables, starts, counts or [T] * B)
    for x, y in zip(bits(cache), bits(want)):
        assert torch.equal(x, y)

    lengths = [min(s + T, n * page) if b % 2 == 0 else s for b, s in enumerate(starts)]
    span = max(lengths) + 3 if max(lengths) + 3 <= n * page else max(lengths)
    gotK, gotV = fa.fa_cache_read(cache, tables, torch.tensor(lengths, dtype=torch.int32, device="cuda"), span)
    p = torch.arange(span, device="cuda")
    for got, pool, scale in ((gotK, cache.K, cache.k_scale), (gotV, cache.V, cache.v_scale)):
        x = pool.view(torch.uint8 if quant else torch.int16)[tables.long()[:, p // page], :, p % page].view(pool.dtype)
        x = x.transpose(1, 2)
        if quant:
            x = (x.float() * scale[tables.long()[:, p // page], :, p % page].transpose(1, 2)[..., None]).to(bf)
        for b, length in enumerate(lengths):
            assert torch.equal(got[b, :, :length].view(torch.int16), x[b, :, :length].contiguous().view(torch.int16))
            assert (got[b, :, length:] == 0).all()
    assert fa.fa_last_device_status() == fa.FA_OK


@pytest.mark.gpu
def test_write_extreme_values():
    """Rows of NaN, infinities, the largest and the smallest values."""
    cache = fa.KVCache.empty(2, 1, 16, 64, dtype=f8)
    x = torch.randn(1, 1, 16, 64, device="cuda").to(bf)
    x[0, 0, 1, 7], x[0, 0, 2, 63], x[0, 0, 3, 0] = math.nan, math.inf, -math.inf
    x[0, 0, 4] = torch.finfo(bf).max
    x[0, 0, 5] = 0
    x[0, 0, 6] *= 2.0 ** -70
    x[0, 0, 7] = -x[0, 0, 8]
    tables = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    fa.fa_cache_write(cache, x, x, tables, torch.zeros(1, dtype=torch.int32, device="cuda"))
    K, V = fa.fa_cache_read(cache, tables, torch.tensor([16], dtype=torch.int32, device="cuda"), 16)
    assert torch.equal(K.view(torch.int16), V.view(torch.int16))
    assert torch.isnan(K[0, 0, 1:4]).all() and (K[0, 0, 5] == 0).all()
    assert (cache.K.view(torch.uint8)[1, 0, 1:4] == 0).all()
    ok = [0] + list(range(4, 16))
    y, a = x[0, 0].double(), x[0, 0].double().abs().amax(-1, keepdim=True)
    # off by half a step of e4m3 (2^-4), of its smallest step (2^-10) below 2^-6 of 448, and half a step of bf16
    tol = 2.0 ** -4 * y.abs() + 2.0 ** -10 / 448 * a.clamp_min(2.0 ** -60) + 2.0 ** -8 * y.abs()
    assert ((K[0, 0].double() - y).abs()[ok] <= tol[ok] * 1.0000002).all()
    assert torch.equal(K[0, 0, 7], -K[0, 0, 8])


@pytest.mark.gpu
def test_bad_tables_reach_no_memory_and_are_reported():
    s = Setup([40, 40], 2, 64, 64, True, 16)
    before = [x.clone() for x in bits(s.cache)]
    tables = s.tables.clone()
    tables[0, 1], tables[1, 2] = -1, 10 ** 6
    x = torch.randn(2, 2, 16, 64, device="cuda").to(bf)
    at = torch.tensor([16, 32], dtype=torch.int32, device="cuda")
    fa.fa_cache_write(s.cache, x, x, tables, at)
    assert fa.fa_last_device_status() == fa.FA_ERR_BAD_TABLE
    assert fa.fa_last_device_status() == fa.FA_OK
    fa.fa_cache_write(s.cache, x, x, s.tables, torch.tensor([-100, 4000], dtype=torch.int32, device="cuda"))
    assert fa.fa_last_device_status() == fa.FA_ERR_BAD_TABLE
    for got, was in zip(bits(s.cache), before):
        assert torch.equal(got.view(torch.uint8), was.view(torch.uint8))
    K, _ = fa.fa_cache_read(s.cache, tables, s.lengths, 40)
    assert fa.fa_last_device_status() == fa.FA_ERR_BAD_TABLE
    assert (K[0, :, 16:32] == 0).all() and (K[1, :, 32:] == 0).all() and (K[1, :, :32] != 0).any()
    Q = query(s, 4, 1)
    good = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths)
    fa.fa_cache_attention(Q, s.cache, tables, s.lengths)
    assert fa.fa_last_device_status() == fa.FA_ERR_BAD_TABLE
    # lengths past the table, groups that are no runs
    fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths + 1000)
    assert fa.fa_last_device_status() == fa.FA_ERR_BAD_TABLE
    for starts in ([0, 3], [2, 0], [-1, 2]):
        O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths,
                                     prefix=(s.tables[:1], s.lengths[:1], torch.tensor(starts, dtype=torch.int32, device="cuda")))
        assert fa.fa_last_device_status() == fa.FA_ERR_BAD_TABLE
    again = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths)
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])
    assert fa.fa_last_device_status() == fa.FA_OK


# ---------------------------------------------------------------- used together (GPU)
@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("mods", [dict(), dict(softcap=30.0, window=50)])
def test_generation_follows_the_forward(mods, quant):
    """A prompt and then single tokens through rotary, write and attention, against fa_forward
    over what the cache holds: the same rows of one causal attention.  The two round
    their weights apart (2^-8 each at most) and their results (2^-8 each)."""
    B, Hq, Hkv, d, prompt, T = 2, 8, 2, 128, 70, 75
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    qkv = torch.randn(B, T, Hq + 2 * Hkv, d, generator=g, device="cuda").to(bf)
    inv = (1e4 ** (-torch.arange(d // 2, device="cuda") * 2.0 / d)).float()
    cache = fa.KVCache.empty(12, Hkv, 32, d, dtype=f8 if quant else bf)
    tables = torch.randperm(12, generator=g, device="cuda")[:6].to(torch.int32).view(B, 3)
    rows, queries = [], []
    at = 0
    while at < T:
        n = prompt if at == 0 else 1
        new = qkv[:, at:at + n]
        pos = torch.arange(at, at + n, device="cuda", dtype=torch.int32)
        Q, K = fa.rotary(new[:, :, :Hq].transpose(1, 2), new[:, :, Hq:Hq + Hkv].transpose(1, 2), pos, inv)
        starts = torch.full((B,), at, dtype=torch.int32, device="cuda")
        fa.fa_cache_write(cache, K, new[:, :, Hq + Hkv:].transpose(1, 2), tables, starts)
        rows.append(fa.fa_cache_attention(Q, cache, tables, starts + n, **mods))
        queries.append(Q)
        at += n
    O, L = torch.cat([r[0] for r in rows], 2), torch.cat([r[1] for r in rows], 2)
    K, V = fa.fa_cache_read(cache, tables, torch.full((B,), T, dtype=torch.int32, device="cuda"), T)
    Q = torch.cat(queries, 2)
    Or, Lr = fa.fa_forward(Q, K, V, True, **mods)
    # read back, a row is rounded to bf16: keys and values are off by another 2^-8 each
    size = torch.einsum("bhqd,bhkd->bhqk", Q.double().abs(), K.double().abs().repeat_interleave(Hq // Hkv, 1)).amax(-1) / d ** 0.5
    off = (2.0 ** -8 * size if quant else 0.0) + d * 2.0 ** -22 * size + 2.0 ** -18 * (1 + mods.get("softcap", 0.0))
    assert ((L - Lr).abs() <= off).all()
    A = V.double().abs().amax(2).repeat_interleave(Hq // Hkv, 1)[:, :, None]
    assert ((O.double() - Or.double()).abs() <= A * ((5 if quant else 4) * 2.0 ** -8 + 2 * off[..., None])).all()


@pytest.mark.gpu
def test_shared_prefix_is_the_same_as_a_copy_for_each():
    """A prefix shared by tables of its own against the same pages in front of every sequence's."""
    s = Setup([33, 64, 1, 90], 2, 128, 128, True, 16, [64])
    Q = query(s, 8, 1)
    O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix)
    tables = torch.cat((s.p_tables[:, :4].expand(4, 4), s.tables), 1).contiguous()
    Oc, Lc = fa.fa_cache_attention(Q, s.cache, tables, s.lengths + 64)
    assert ((L - Lc).abs() <= 2.0 ** -18 * (1 + L.abs())).all()
    # weights are rounded against other references: 2^-11 each, and both results
    top = max(float(x.abs().max()) for x in fa.fa_cache_read(s.cache, tables, s.lengths + 64, 154)[1:])
    assert ((O.double() - Oc.double()).abs() <= 2.0 ** -10 * top + 2.0 ** -7 * O.double().abs()).all()


@pytest.mark.gpu
def test_captured_step_is_replayed_with_other_lengths():
    """Write and attention in one graph: the next tokens, lengths and pages are what the
    buffers hold at the replay; two graphs with one workspace, replayed in turn."""
    s = Setup([102, 32, 61], 2, 64, 64, True, 16, extra_cols=60)  # (all that a replay sees is held: the rest is NaN)
    K, V = (torch.randn(3, 2, 1, 64, device="cuda").to(bf) for _ in range(2))
    Q, starts = query(s, 4, 1), torch.tensor([100, 30, 7], dtype=torch.int32, device="cuda")
    lengths = starts + 1
    ws = torch.empty(fa.fa_cache_attention_workspace_bytes(Q, s.cache, s.tables), dtype=torch.uint8, device="cuda")

    def step():
        fa.fa_cache_write(s.cache, K, V, s.tables, starts)
        torch.add(starts, 1, out=lengths)
        return fa.fa_cache_attention(Q, s.cache, s.tables, lengths, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for k, new in enumerate(([100, 30, 7], [101, 31, 8], [17, 0, 60])):
        starts.copy_(torch.tensor(new, dtype=torch.int32))
        K.normal_()
        graph, (O, L) = graphs[k % 2]
        graph.replay()
        torch.cuda.synchronize()
        s.lens = [n + 1 for n in new]
        check(s, Q, O, L)


@pytest.mark.gpu
def test_two_streams_at_once():
    a = Setup([3000] * 8, 4, 128, 128, True, 64, seed=1)
    b = Setup([1000] * 5, 2, 64, 64, False, 16, [700], seed=2)
    Qa, Qb = query(a, 16, 1), query(b, 4, 2)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        Oa, La = fa.fa_cache_attention(Qa, a.cache, a.tables, a.lengths, stream=streams[0])
        Ob, Lb = fa.fa_cache_attention(Qb, b.cache, b.tables, b.lengths, prefix=b.prefix, stream=streams[1])
    K, V = fa.fa_cache_read(b.cache, b.tables, b.lengths, 1000, stream=streams[1])
    torch.cuda.synchronize()
    check(a, Qa, Oa, La)
    check(b, Qb, Ob, Lb)
    assert torch.equal(K[0].double(), b.rows(b.tables[0], 1000)[0])


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes (and, of the scales, 2^31): its last pages are used."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    pages = (1 << 32) // (8 * 256 * 64) + 40
    raw = [torch.empty(pages, 8, 256, 64, dtype=torch.uint8, device="cuda").view(f8) for _ in range(2)]
    cache = fa.KVCache(*raw, *(torch.empty(pages, 8, 256, device="cuda") for _ in range(2)))
    tables = torch.tensor([[pages - 1, pages - 3], [2, pages - 2]], dtype=torch.int32, device="cuda")
    K, V = (torch.randn(2, 8, 300, 64, device="cuda").to(bf) for _ in range(2))
    fa.fa_cache_write(cache, K, V, tables, torch.zeros(2, dtype=torch.int32, device="cuda"))
    lengths = torch.tensor([300, 290], dtype=torch.int32, device="cuda")
    gotK, gotV = fa.fa_cache_read(cache, tables, lengths, 300)
    for got, x in ((gotK, K), (gotV, V)):
        codes, a = quantise(x)
        want = (codes.float() * a[..., None]).to(bf)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1, :, :290], want[1, :, :290])
    Q = torch.randn(2, 16, 1, 64, device="cuda").to(bf)
    s = Setup([1, 1], 8, 64, 64, True, 256)
    s.cache, s.tables, s.lengths, s.lens = cache, tables, lengths, [300, 290]
    check(s, Q, *fa.fa_cache_attention(Q, cache, tables, lengths))
