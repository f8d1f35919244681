"""Attention with modified scores (cap, distance slopes) and planned masks
(documents, prefixes): the CUDA path against the definition in float64, and
the refusals of bad arguments.

Tolerances.  O, dQ, dK, dV: rel-L2 1e-2 (tests/parity.py), and for each element
the sum of what its terms can be off by, with half a bf16 step r = 2^-8 for each
rounding and e = 2^-12 + 2^-20 c for the fp32 weights (scores off as L is, below):
    O_i   r |O_i| + sum_j (r + e) P_ij |V_j|                 (P is rounded to bf16)
    dV_j  r |dV_j| + sum_i (r + e) P_ij |dO_i|
    dx_ij off by  (r + e) |dx_ij| + P_ij t_ij d_i, with D = rowsum(dO O) off by
          d_i = sum_c (r |O_ic| + its own bound) |dO_ic|     (O is rounded to bf16),
          t the cap's derivative, and by 2^-21 P_ij |dP_ij - D_i| with a cap: t is
          4 w (1 - w) with w = 1 / (1 + exp(2x/c)) <= 1 in fp32, where the sum and
          the reciprocal are each off by 2^-24 of w, so 1 - w is by 2^-23 near w = 1
    dQ_i  r |dQ_i| + scale sum_j (dx_ij's) |K_j|,  dK_j likewise with |Q_i|.
    and 2^-100 where weights underflow (P below 2^-126 counts as 0: at most 2^13
    terms of values up to 2^8 each).
(The 2e-2 of tests/parity.py is for inputs of unit size, its element-wise bar does
not follow the inputs' size: a dK of Q eight times as large is off by eight times
as much.)  L (fp32) <= 1e-4 + 2^-20 c: a product of
128 terms of |q||k| <= 5 * 5 summed in fp32 is off by at most
128 * 2^-24 * 25 * sqrt(128) / sqrt(128) ~ 2e-4 / 11 after the 1/sqrt(d), the
exponentials and the logarithm add 1e-6.  A cap c adds 2^-20 c: x = c (1 - 2 r)
with r <= 1 off by 9 steps of 2^-24 (ex2 2^-22 on half of the sum, the sum, five
products for the reciprocal shared by four scores 2^-24 each, rcp 2^-23)."""
import ctypes
import math

import pytest
import torch

import tiled_attention_05_gb300 as fa
from tests.parity import assert_close

bf = torch.bfloat16


# ---------------------------------------------------------------- definition in float64
def visible(B, Tq, Tk, causal, window=0, doc_q=None, doc_k=None, prefix=None, device="cpu"):
    i = torch.arange(Tq, device=device)[:, None] + Tk - Tq
    j = torch.arange(Tk, device=device)[None, :]
    v = (j <= i) if causal else torch.ones(Tq, Tk, dtype=torch.bool, device=device)
    v = v.expand(B, Tq, Tk)
    if prefix is not None:
        v = v | (j < (prefix[:, None, None] if prefix.dim() == 1 else prefix[:, :, None]))
    if window:
        v = v & (j > i - window)
    if doc_q is not None:
        v = v & (doc_q[:, :, None] == doc_k[:, None, :]) & (doc_q >= 0)[:, :, None]
    return v


def definition(Q, K, V, vis, softcap=0.0, slopes=None, scale=None, more=False):
    """O, L in the dtype of Q, K, V, differentiable (``more``: also P and the
    cap's derivative)."""
    B, Hq, Tq, d = Q.shape
    G, Tk = Hq // K.shape[1], K.shape[2]
    K, V = K.repeat_interleave(G, 1), V.repeat_interleave(G, 1)
    x = torch.matmul(Q, K.transpose(2, 3)) * (scale or d ** -0.5)
    slope = None
    if softcap:
        t = torch.tanh(x / softcap)
        x, slope = softcap * t, 1 - t.detach() ** 2
    if slopes is not None:
        far = (torch.arange(Tq, device=Q.device)[:, None] + Tk - Tq - torch.arange(Tk, device=Q.device)).abs()
        x = x - slopes.to(x.dtype)[:, None, None] * far
    vis = vis[:, None]
    m = x.detach().masked_fill(~vis, -math.inf).amax(-1, keepdim=True) if Tk else x.new_zeros(B, Hq, Tq, 1)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(torch.where(vis, x - m, -1e4)) * vis
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, 1.0)
    O, L = torch.matmul(p, V), (m + torch.log(l)).squeeze(-1)
    return (O, L, p.detach(), slope) if more else (O, L)


def element_bounds(Q, K, V, dO, O, P, slope, grads, scale, cap):
    """How far each element of O, dQ, dK, dV may be off (see the module's head)."""
    r, e = 2.0 ** -8, 2.0 ** -12 + 2.0 ** -20 * cap
    B, Hq, Tq, d = Q.shape
    Hkv, Tk = K.shape[1], K.shape[2]
    G = Hq // Hkv
    q, g, o = Q.double().abs(), dO.double().abs(), O.double().abs()
    k, v = (t.double().repeat_interleave(G, 1) for t in (K, V))
    group = lambda t: t.unflatten(1, (Hkv, G)).sum(2)  # noqa: E731
    bO = r * o + (r + e) * torch.matmul(P, v.abs())
    off_D = ((r * o + bO) * g).sum(-1, keepdim=True)
    dP = torch.matmul(dO.double(), v.transpose(2, 3))
    dx = P * (dP - (O.double() * dO.double()).sum(-1, keepdim=True))
    w, off_x = P, 0.0
    if slope is not None:
        off_x = 2.0 ** -21 * dx.abs()
        dx, w = dx * slope, P * slope
    off_x = off_x + (r + e) * dx.abs() + w * off_D
    scale = scale or d ** -0.5
    dQ, dK, dV = (t.abs() for t in grads)
    return (bO, r * dQ + scale * torch.matmul(off_x, k.abs()),
            r * dK + scale * group(torch.matmul(off_x.transpose(2, 3), q)),
            r * dV + (r + e) * group(torch.matmul(P.transpose(2, 3), g)))


def inputs(B, Hq, Hkv, Tq, Tk, d, dv, seed, device="cuda", std=1.0):
    g = torch.Generator(device).manual_seed(seed)
    draw = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    return ((std * draw(B, Hq, Tq, d)).to(bf), draw(B, Hkv, Tk, d).to(bf), draw(B, Hkv, Tk, dv).to(bf),
            draw(B, Hq, Tq, dv).to(bf))


def alibi(H, device="cuda"):
    return (2.0 ** (-8.0 * torch.arange(1, H + 1, dtype=torch.float64) / H)).float().to(device)


def compare(Q, K, V, dO, causal, window=0, softcap=0.0, slopes=None, docs=None, prefix=None, scale=None, tag=""):
    doc_q, doc_k = docs if docs is not None else (None, None)
    B, Hq, Tq, _ = Q.shape
    Tk = K.shape[2]
    mask = None
    if docs is not None or prefix is not None:
        mask = fa.fa_mask_plan(B, Tq, Tk, causal, window, doc_q, doc_k, prefix)
    mods = dict(window=window, softcap=softcap, slopes=slopes, mask=mask)
    O, L = fa.fa_forward(Q, K, V, causal, scale, **mods)
    dQ, dK, dV = fa.fa_backward(Q, K, V, O, dO, L, causal, scale, **mods)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == fa.FA_OK
    vis = visible(B, Tq, Tk, causal, window, doc_q, doc_k, prefix, Q.device)
    q, k, v = (t.double().requires_grad_() for t in (Q, K, V))
    Or, Lr, P, slope = definition(q, k, v, vis, softcap, slopes, scale, more=True)
    grads = torch.autograd.grad(Or, (q, k, v), dO.double())
    Lr = Lr.detach()
    off = torch.where(torch.isinf(Lr) & (L == Lr), 0.0, (L - Lr).abs())  # -inf where -inf is due
    assert not off.numel() or float(off.max()) <= 1e-4 + 2.0 ** -20 * softcap, (tag, "L", float(off.max()))
    refs = (Or.detach(),) + grads
    bounds = element_bounds(Q, K, V, dO, refs[0], P, slope, grads, scale, softcap)
    for name, got, ref, bound in zip(("O", "dQ", "dK", "dV"), (O, dQ, dK, dV), refs, bounds):
        if not ref.numel():
            continue
        off = (got.double() - ref).abs()
        assert bool((off <= bound + 2.0 ** -100).all()), (tag, name, float((off - bound).max()), float(off.max()))
        if float(ref.norm()) > 2 * float(bound.norm()):  # else rounding is all there is
            assert float(off.norm()) <= 1e-2 * float(ref.norm()), (tag, name, float(off.norm() / ref.norm()))
    hidden = ~vis.any(-1)[:, None].expand(B, Hq, Tq)  # rows that see nothing
    assert bool((O[hidden] == 0).all()) and bool((dQ[hidden] == 0).all()) and bool((L[hidden] == -math.inf).all())
    return O, L, dQ, dK, dV


# ---------------------------------------------------------------- refusals (CPU)
def cpu(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refusals():
    Q, K, V = cpu(1, 4, 10, 64), cpu(1, 2, 10, 64), cpu(1, 2, 10, 64)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        fa.fa_forward(Q, K, V, True, softcap=30.0)
    ids = cpu(1, 10, dtype=torch.int32)
    with pytest.raises(ValueError, match="go together"):
        fa.fa_mask_plan(1, 10, 10, True, doc_q=ids)
    with pytest.raises(ValueError, match="documents or a prefix"):
        fa.fa_mask_plan(1, 10, 10, True)
    with pytest.raises(ValueError, match="doc_k has shape"):
        fa.fa_mask_plan(1, 10, 9, True, doc_q=ids, doc_k=ids)
    with pytest.raises(ValueError, match="contiguous CUDA torch.int32"):
        fa.fa_mask_plan(1, 10, 10, True, doc_q=ids.long(), doc_k=ids.long())
    with pytest.raises(ValueError, match="prefix has shape"):
        fa.fa_mask_plan(1, 10, 10, True, prefix=cpu(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="prefix has shape"):
        fa.fa_mask_plan(1, 10, 10, True, prefix=cpu(1, 1, 10, dtype=torch.int32))
    with pytest.raises(ValueError, match="B, H, T, d"):
        fa.attention(Q[0], K, V, docs=ids)
    with pytest.raises(ValueError, match="plan already"):
        fa.attention(Q, K, V, docs=ids, mask=fa.MaskPlan((1, 10, 10, 0, 0), ids))
    dims = fa.make_dims(1, 4, 2, 10, 10, 64, 64, True, None)
    with pytest.raises(ValueError, match="was planned for"):
        fa._scores(dims, torch.device("cpu"), 0.0, None, fa.MaskPlan((1, 10, 11, 1, 0), ids), None)
    with pytest.raises(ValueError, match="must be a MaskPlan"):
        fa._scores(dims, torch.device("cpu"), 0.0, None, ids, None)
    with pytest.raises(ValueError, match="no gradient"):
        fa._scores(dims, torch.device("cpu"), 0.0, torch.zeros(4, requires_grad=True), None, None)
    with pytest.raises(ValueError, match="slopes has shape"):
        fa._scores(dims, torch.device("cpu"), 0.0, torch.zeros(2), None, None)
    assert fa._scores(dims, torch.device("cpu"), 0.0, None, None, None) is None


P = [0x1000 * (k + 1) for k in range(9)]


def abi(dims, scores):
    lib = fa.load()
    ws = fa.fa_backward_workspace_bytes(dims)
    return {lib.fa_forward_scored(ctypes.byref(dims), ctypes.byref(scores), *P[:5], None, 0, None),
            lib.fa_backward_scored(ctypes.byref(dims), ctypes.byref(scores), *P, 0x100000, ws, 7, None)}


@pytest.mark.parametrize("bad", [dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
                                 dict(softcap=1e-4), dict(softcap=1025.0), dict(slopes=0x1002), dict(plan=0x1008)])
def test_abi_refuses_bad_scores(bad):
    s = fa.FaScores(bad.get("softcap", 0.0), bad.get("slopes"), bad.get("plan"))
    assert abi(fa.make_dims(1, 4, 2, 100, 90, 64, 64, True, None), s) == {fa.FA_ERR_INVALID_ARG}


def test_abi_refuses_distances_past_fp32():
    s = fa.FaScores(0.0, 0x1000, None)
    assert abi(fa.make_dims(1, 1, 1, 100, (1 << 24) + 1, 64, 64, False, None), s) == {fa.FA_ERR_UNSUPPORTED}


def test_abi_refuses_bad_plans():
    lib = fa.load()
    d = fa.make_dims(2, 1, 1, 300, 300, 64, 64, True, None)
    w = fa.make_dims(2, 1, 1, 300, 300, 64, 64, True, None, 100)
    free = fa.make_dims(2, 1, 1, 300, 300, 64, 64, False, None)
    need = lib.fa_mask_plan_bytes(ctypes.byref(d))
    assert need >= 4 * 2 * 6 * 384
    call = lambda dims, *a: lib.fa_mask_plan(ctypes.byref(dims), *a, None)  # noqa: E731
    bad = fa.FA_ERR_INVALID_ARG
    assert call(d, 0x1000, None, None, 0, 0x2000, need) == bad        # one side's documents only
    assert call(d, 0x1000, 0x1002, None, 0, 0x2000, need) == bad      # misaligned
    assert call(d, 0x1000, 0x1000, None, 2, 0x2000, need) == bad      # flag
    assert call(d, 0x1000, 0x1000, None, 0, 0x2000, need - 1) == bad  # too small
    assert call(d, 0x1000, 0x1000, None, 0, 0x2008, need) == bad
    assert call(d, 0x1000, 0x1000, None, 0, None, need) == bad
    assert call(w, None, None, 0x1000, 0, 0x2000, need) == bad        # prefix with a window
    assert call(free, None, None, 0x1000, 0, 0x2000, need) == bad     # prefix without the causal mask
    assert lib.fa_mask_plan(None, None, None, None, 0, None, 0, None) == bad
    assert call(fa.make_dims(0, 1, 1, 300, 300, 64, 64, True, None), None, None, None, 0, None, 0) == fa.FA_OK
    assert lib.fa_mask_plan_bytes(ctypes.byref(fa.make_dims(-1, 1, 1, 3, 3, 64, 64, True, None))) == 0


def test_scores_and_plan_argument_structs_match_the_header():
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fa.h")).read()
    for name, cls in (("fa_scores", fa.FaScores), ("fa_rotary_dims", fa.FaRotaryDims)):
        body = text[:text.index("} %s;" % name)].rsplit("typedef struct {", 1)[1]
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = [re.sub(r"\[\d+\]", "", n).strip(" *\n") for decl in body.split(";") if decl.strip()
                  for n in re.sub(r"^\s*(const\s+)?(long long|int|float|void)\s*\*?", "", decl).split(",")]
        assert fields == [f[0] for f in cls._fields_], name


# ---------------------------------------------------------------- parity (GPU)
gpu = pytest.mark.gpu

# B, Hq, Hkv, Tq, Tk, d, dv, causal, window
SHAPES = [
    (1, 1, 1, 1, 1, 64, 64, True, 0),
    (1, 2, 1, 1, 300, 128, 128, True, 0),        # one new token
    (2, 4, 2, 129, 129, 64, 64, True, 0),
    (1, 4, 4, 300, 257, 128, 64, True, 0),       # more rows than keys: the first see nothing
    (1, 4, 1, 200, 520, 64, 128, True, 70),
    (2, 2, 2, 260, 130, 128, 128, False, 0),
    (1, 3, 1, 384, 640, 64, 64, False, 0),
    (1, 2, 2, 600, 600, 128, 128, True, 128),
]
SCORES = [("cap", 20.0, False), ("slopes", 0.0, True), ("both", 50.0, True)]


@gpu
@pytest.mark.parametrize("score", SCORES, ids=lambda s: s[0])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_scores(shape, score):
    B, Hq, Hkv, Tq, Tk, d, dv, causal, window = shape
    _, cap, slopes = score
    Q, K, V, dO = inputs(B, Hq, Hkv, Tq, Tk, d, dv, seed=sum(shape), std=2.0)
    compare(Q, K, V, dO, causal, window, cap, alibi(Hq) if slopes else None)


@gpu
@pytest.mark.parametrize("cap, std, scale", [(5.0, 8.0, None), (2.0 ** -10, 1.0, None), (1000.0, 1.0, None),
                                             (1024.0, 1.0, 0.3), (30.0, 1.0, 4.0)])
def test_caps_from_saturated_to_idle(cap, std, scale):
    Q, K, V, dO = inputs(1, 2, 1, 200, 200, 64, 64, seed=9, std=std)
    compare(Q, K, V, dO, True, softcap=cap, scale=scale)


@gpu
def test_slopes_of_any_sign_and_zero():
    Q, K, V, dO = inputs(1, 4, 2, 300, 300, 64, 64, seed=10)
    slopes = torch.tensor([0.0, -0.02, 3.0, 40.0], device="cuda")
    compare(Q, K, V, dO, True, slopes=slopes)
    compare(Q, K, V, dO, False, slopes=slopes.abs())


def packed(B, T, seed, pad=True, tile_edges=False):
    """Ascending document ids of a packed row, padding last."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.full((B, T), -1, dtype=torch.int32)
    for b in range(B):
        at, n = 0, 3 * b
        while at < T - (T // 7 if pad else 0):
            k = 128 if tile_edges else int(torch.randint(1, max(2, T // 3), (1,), generator=g))
            ids[b, at:at + k] = n
            at, n = at + k, n + 1 + int(torch.randint(0, 2, (1,), generator=g))
    return ids.cuda()


DOC_SHAPES = [(1, 2, 1, 1, 64, 64), (2, 4, 2, 300, 64, 64), (1, 4, 1, 777, 128, 128), (2, 2, 2, 512, 128, 64),
              (1, 6, 2, 1100, 64, 128)]


@gpu
@pytest.mark.parametrize("score", [("mask", 0.0, False)] + SCORES, ids=lambda s: s[0])
@pytest.mark.parametrize("shape", DOC_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_packed_documents(shape, score):
    B, Hq, Hkv, T, d, dv = shape
    _, cap, slopes = score
    Q, K, V, dO = inputs(B, Hq, Hkv, T, T, d, dv, seed=sum(shape) + 1)
    ids = packed(B, T, seed=T)
    for causal, window in ((True, 0), (False, 0), (True, max(1, T // 9))):
        compare(Q, K, V, dO, causal, window, cap, alibi(Hq) if slopes else None, docs=(ids, ids),
                tag=f"causal {causal} window {window}")


@gpu
@pytest.mark.parametrize("kind", ["tile_edges", "one", "all_padding", "every_token", "left_padding", "shuffled",
                                  "interleaved", "huge_ids", "descending"])
@pytest.mark.parametrize("causal", [True, False])
def test_documents_in_every_order(kind, causal):
    B, T = 2, 515
    g = torch.Generator().manual_seed(4)
    ids = {
        "tile_edges": lambda: packed(B, T, 1, pad=False, tile_edges=True).cpu(),
        "one": lambda: torch.full((B, T), 7),
        "all_padding": lambda: torch.stack((torch.full((T,), -5), torch.arange(T) // 100)),
        "every_token": lambda: torch.arange(T).expand(B, T),
        "left_padding": lambda: (torch.arange(T) // 150 - 1).expand(B, T),
        "shuffled": lambda: torch.randint(-1, 5, (B, T), generator=g),
        "interleaved": lambda: torch.stack((torch.arange(T) % 3, torch.arange(T) // 200 % 2)),
        "huge_ids": lambda: (2 ** 31 - 1 - torch.arange(T).flip(0) // 170).expand(B, T),  # the last one is padding
        "descending": lambda: (torch.arange(T).flip(0) // 90).expand(B, T),
    }[kind]().to(torch.int32).cuda().contiguous()
    Q, K, V, dO = inputs(B, 2, 1, T, T, 64, 64, seed=8)
    docs = torch.where(ids == 2 ** 31 - 1, -1, ids)  # as documented: 2^31 - 1 is padding too
    mask = fa.fa_mask_plan(B, T, T, causal, 0, ids, ids)
    O, L = fa.fa_forward(Q, K, V, causal, mask=mask)
    O2, L2, *_ = compare(Q, K, V, dO, causal, docs=(docs, docs), tag=kind)
    assert torch.equal(O, O2) and torch.equal(L, L2)


@gpu
@pytest.mark.parametrize("Tq, Tk", [(300, 700), (700, 300), (1, 400), (400, 1), (128, 1024), (513, 129)])
def test_documents_of_other_rows_than_keys(Tq, Tk):
    B = 2
    doc_k = packed(B, Tk, 5)
    g = torch.Generator().manual_seed(6)
    some = torch.randint(-1, int(doc_k.max()) + 2, (B, Tq), generator=g, dtype=torch.int32).cuda()
    Q, K, V, dO = inputs(B, 2, 2, Tq, Tk, 64, 128, seed=Tq)
    for doc_q in (some, some.sort(-1).values):
        for causal in (True, False):
            compare(Q, K, V, dO, causal, softcap=30.0, docs=(doc_q, doc_k), tag=f"causal {causal}")


@gpu
@pytest.mark.parametrize("shape", [(2, 4, 2, 300, 300, 64, 64), (3, 2, 1, 200, 450, 128, 128), (2, 2, 2, 450, 200, 64, 128),
                                   (2, 2, 1, 1, 1, 64, 64)], ids=lambda s: "x".join(map(str, s)))
def test_prefix(shape):
    B, Hq, Hkv, Tq, Tk, d, dv = shape
    Q, K, V, dO = inputs(B, Hq, Hkv, Tq, Tk, d, dv, seed=sum(shape))
    g = torch.Generator().manual_seed(7)
    for prefix in (torch.tensor([0, Tk, Tk // 2][:B]), torch.tensor([-3, Tk + 99, 130][:B]),
                   torch.randint(0, Tk + 1, (B, Tq), generator=g),            # a prefix of its own for each row
                   torch.full((B, Tq), 140).where(torch.arange(Tq) < 140, 0)):
        p = prefix.to(torch.int32).cuda()
        compare(Q, K, V, dO, True, prefix=p)
        compare(Q, K, V, dO, True, softcap=25.0, slopes=alibi(Hq), prefix=p)


@gpu
def test_prefix_of_each_packed_document():
    B, T = 1, 600
    ids = (torch.arange(T) // 200).to(torch.int32).cuda()[None]
    prefix = (ids * 200 + 60).contiguous()  # the first 60 tokens of each document see each other
    Q, K, V, dO = inputs(B, 4, 2, T, T, 128, 128, seed=3)
    compare(Q, K, V, dO, True, docs=(ids, ids), prefix=prefix)


def same_up_to_order(got, want):
    """The same P (its reference does not depend on the split), fp32 sums in another
    order, rounded once: one bf16 step of each element (and 1e-4 near zero, where
    terms of both signs met), 1e-5 of L."""
    (O, L), (O2, L2) = got[:2], want[:2]
    assert float((L - L2).abs().max()) <= 1e-5
    assert bool(((O.float() - O2.float()).abs() <= 2.0 ** -7 * O2.float().abs() + 1e-4).all())


@gpu
def test_one_document_is_the_plain_call():
    for B in (1, 8):
        Q, K, V, dO = inputs(B, 4, 2, 700, 700, 128, 128, seed=2)
        ids = torch.zeros(B, 700, dtype=torch.int32, device="cuda")
        O, L, *_ = compare(Q, K, V, dO, True, docs=(ids, ids))
        if B > 1:  # (one batch row is few enough work to be split over the keys: other references of P, other rounding)
            want = fa.fa_forward(Q, K, V, True)
            assert torch.equal(O, want[0]) and torch.equal(L, want[1])


@gpu
@pytest.mark.parametrize("score", [("mask", 0.0, False)] + SCORES, ids=lambda s: s[0])
def test_a_row_of_one_key_returns_its_value(score):
    _, cap, slopes = score
    B, H, T, d = 1, 4, 900, 64
    Q, K, V, dO = inputs(B, H, H, T, T, d, d, seed=5)
    ids = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    mask = fa.fa_mask_plan(B, T, T, True, 0, ids, ids)  # every token a document
    O, L = fa.fa_forward(Q, K, V, True, softcap=cap, slopes=alibi(H) if slopes else None, mask=mask)
    assert torch.equal(O, V)
    O, L = fa.fa_forward(Q[:, :, :1].contiguous(), K[:, :, :1].contiguous(), V[:, :, :1].contiguous(), True,
                         softcap=cap or 9.0, slopes=alibi(H) if slopes else None)
    assert torch.equal(O, V[:, :, :1])


@gpu
def test_empty_sizes():
    z = lambda *s: torch.zeros(*s, device="cuda", dtype=bf)  # noqa: E731
    ids = lambda T: torch.zeros(1, T, device="cuda", dtype=torch.int32)  # noqa: E731
    for Tq, Tk in ((5, 0), (0, 5), (0, 0)):
        mask = fa.fa_mask_plan(1, Tq, Tk, True, 0, ids(Tq), ids(Tk))
        Q, K, V = z(1, 2, Tq, 64), z(1, 2, Tk, 64), z(1, 2, Tk, 64)
        O, L = fa.fa_forward(Q, K, V, True, softcap=5.0, slopes=alibi(2), mask=mask)
        dQ, dK, dV = fa.fa_backward(Q, K, V, O, O, L, True, softcap=5.0, slopes=alibi(2), mask=mask)
        assert not O.any() and not dQ.any() and not dK.any() and not dV.any() and bool((L == -math.inf).all())
    fa.fa_mask_plan(0, 5, 5, True, 0, torch.zeros(0, 5, device="cuda", dtype=torch.int32),
                    torch.zeros(0, 5, device="cuda", dtype=torch.int32))


# few rows over many keys: heads packed into one tile, key tiles split over the SMs
@gpu
@pytest.mark.parametrize("shape", [(1, 8, 2, 32, 8032, 128, 128), (2, 4, 1, 1, 5000, 64, 64), (1, 8, 1, 64, 2100, 64, 128),
                                   (3, 2, 2, 7, 1500, 128, 64), (1, 32, 1, 40, 700, 128, 128), (1, 4, 2, 300, 3000, 64, 64),
                                   (1, 6, 2, 65, 1000, 64, 64)], ids=lambda s: "x".join(map(str, s)))
def test_few_rows(shape):
    B, Hq, Hkv, Tq, Tk, d, dv = shape
    Q, K, V, dO = inputs(B, Hq, Hkv, Tq, Tk, d, dv, seed=sum(shape))
    g = torch.Generator().manual_seed(1)
    doc_k, some = packed(B, Tk, 9), torch.randint(0, 4, (B, Tk), generator=g, dtype=torch.int32).cuda()
    rows = doc_k[:, -Tq:].contiguous().clamp(min=0)
    prefix = torch.full((B,), Tk // 3, dtype=torch.int32, device="cuda")
    for name, cap, slopes in SCORES + [("wide cap", 200.0, True)]:
        slopes = alibi(Hq) if slopes else None
        compare(Q, K, V, dO, True, 0, cap, slopes, tag=name)
        compare(Q, K, V, dO, True, Tk // 2, cap, slopes, tag=name + " window")
        compare(Q, K, V, dO, False, 0, cap, slopes, tag=name + " full")
        compare(Q, K, V, dO, True, 0, cap, slopes, docs=(rows, doc_k), tag=name + " documents")
        compare(Q, K, V, dO, False, 0, cap, slopes, docs=(some[:, :Tq].contiguous(), some), tag=name + " any order")
        compare(Q, K, V, dO, True, 0, cap, slopes, prefix=prefix, tag=name + " prefix")
    compare(Q, K, V, dO, False, 0, 0.0, None, docs=(rows, doc_k), tag="documents alone")
    # heads of one tile with gentle, steep and negative slopes
    mixed = torch.tensor([0.05, 20.0, -0.01, 7.0], device="cuda").repeat(-(-Hq // 4))[:Hq].contiguous()
    for cap in (0.0, 30.0, 200.0):
        compare(Q, K, V, dO, True, 0, cap, mixed, tag=f"mixed slopes, cap {cap}")


@gpu
def test_the_split_workspace_is_optional():
    B, Hq, Hkv, Tq, Tk, d = 1, 8, 2, 32, 4000, 128
    Q, K, V, dO = inputs(B, Hq, Hkv, Tq, Tk, d, d, seed=4)
    dims, lib = fa.make_dims(B, Hq, Hkv, Tq, Tk, d, d, True, None), fa.load()
    scores = fa.FaScores(30.0, None, None)
    need = lib.fa_forward_scored_workspace_bytes(ctypes.byref(dims), ctypes.byref(scores))
    assert need > 0
    assert lib.fa_forward_scored_workspace_bytes(ctypes.byref(dims), ctypes.byref(fa.FaScores(0.0, None, None))) == 0
    want = fa.fa_forward(Q, K, V, True, softcap=30.0)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    for ptr, n, launches in ((None, 0, 1), (ws.data_ptr(), need - 1, 1), (ws.data_ptr(), need, 2)):
        O, L = torch.full_like(Q, 9.0), torch.full((B, Hq, Tq), 9.0, device="cuda")
        code = lib.fa_forward_scored(ctypes.byref(dims), ctypes.byref(scores), Q.data_ptr(), K.data_ptr(), V.data_ptr(),
                                     O.data_ptr(), L.data_ptr(), ptr, n, torch.cuda.current_stream().cuda_stream)
        assert code == fa.FA_OK and fa.last_launch_count() == launches
        same_up_to_order((O, L), want)
    assert lib.fa_forward_scored(ctypes.byref(dims), ctypes.byref(scores), Q.data_ptr(), K.data_ptr(), V.data_ptr(),
                                 O.data_ptr(), L.data_ptr(), ws.data_ptr() + 16, need, None) == fa.FA_ERR_INVALID_ARG


@gpu
def test_random_problems():
    rnd = __import__("random").Random(20)
    for trial in range(40):
        B, Hkv, G = rnd.choice((1, 2)), rnd.choice((1, 2)), rnd.choice((1, 3))
        Tk = rnd.randrange(1, 900)
        Tq = rnd.choice((Tk, Tk, rnd.randrange(1, 900)))
        d, dv = rnd.choice((64, 128)), rnd.choice((64, 128))
        causal = rnd.random() < 0.7
        window = rnd.randrange(1, Tk + 50) if causal and rnd.random() < 0.4 else 0
        cap = rnd.choice((0.0, 15.0, 50.0))
        slopes = alibi(Hkv * G) if rnd.random() < 0.5 else None
        docs = prefix = None
        if rnd.random() < 0.5:
            doc_k = packed(B, Tk, trial)
            docs = (doc_k, doc_k) if Tq == Tk else (packed(B, Tq, trial + 1), doc_k)
        if causal and not window and rnd.random() < 0.4:
            prefix = torch.randint(0, Tk + 1, (B,), generator=torch.Generator().manual_seed(trial)).int().cuda()
        Q, K, V, dO = inputs(B, Hkv * G, Hkv, Tq, Tk, d, dv, seed=trial)
        compare(Q, K, V, dO, causal, window, cap, slopes, docs, prefix,
                tag=f"trial {trial} {(B, Hkv, G, Tq, Tk, d, dv, causal, window, cap)}")


@gpu
def test_gradient_against_differences():
    """<gradient, direction> against central differences of the float64 loss."""
    B, H, T, d = 1, 2, 150, 64
    Q, K, V, dO = inputs(B, H, H, T, T, d, d, seed=11)
    ids = packed(B, T, 3)
    vis = visible(B, T, T, True, 0, ids, ids, None, "cuda")
    slopes = alibi(H)
    mask = fa.fa_mask_plan(B, T, T, True, 0, ids, ids)
    O, L = fa.fa_forward(Q, K, V, True, softcap=10.0, slopes=slopes, mask=mask)
    grads = fa.fa_backward(Q, K, V, O, dO, L, True, softcap=10.0, slopes=slopes, mask=mask)
    xs = [t.double() for t in (Q, K, V)]
    g = torch.Generator("cuda").manual_seed(12)
    for k in range(3):
        way = torch.randn(xs[k].shape, generator=g, device="cuda", dtype=torch.float64)
        loss = lambda h: float((definition(*[x + h * way if n == k else x for n, x in enumerate(xs)], vis, 10.0,  # noqa: E731
                                           slopes)[0] * dO.double()).sum())
        want = (loss(1e-5) - loss(-1e-5)) / 2e-5
        got = float((grads[k].double() * way).sum())
        # rel-L2 1e-2 of the gradient, met by an independent unit direction: 1e-2 |g| times a normal variate, below 5
        assert abs(got - want) <= 5e-2 * float(grads[k].double().norm()), (k, got, want)


@gpu
def test_autograd_layer_of_rotary_and_documents():
    """A training layer: packed projection -> rotary -> capped attention over
    packed documents -> gradients, against the same in float64."""
    B, T, Hq, Hk, d = 2, 333, 4, 2, 64
    g = torch.Generator("cuda").manual_seed(13)
    qkv = torch.randn(B, T, Hq + 2 * Hk, d, generator=g, device="cuda").to(bf).requires_grad_()
    dO = torch.randn(B, Hq, T, d, generator=g, device="cuda").to(bf)
    ids = packed(B, T, 2)
    pos = torch.randint(0, 3000, (3, B, T), generator=g, device="cuda", dtype=torch.int32)
    f = (1e4 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()

    def layer(qkv, attend, turn):
        q, k, v = (t.transpose(1, 2) for t in qkv.split((Hq, Hk, Hk), 2))
        q, k = turn(q, k)
        return attend(q, k, v)

    def turn64(q, k):
        axis = [0] * 10 + [1] * 12 + [2] * 10
        th = torch.stack([pos[a].double() * f[n].double() for n, a in enumerate(axis)], -1)[:, None]
        c, s = th.cos(), th.sin()
        return [torch.cat((x[..., :32] * c - x[..., 32:] * s, x[..., 32:] * c + x[..., :32] * s), -1) for x in (q, k)]

    vis = visible(B, T, T, True, 0, ids, ids, None, "cuda")
    x = qkv.detach().double().requires_grad_()
    Or = layer(x, lambda q, k, v: definition(q, k, v, vis, 20.0, alibi(Hq))[0], turn64)
    gr, = torch.autograd.grad(Or, x, dO.double())
    plan = fa.fa_mask_plan(B, T, T, True, 0, ids, ids)
    turn = lambda q, k: fa.rotary(q, k, pos, f, (10, 12, 10))  # noqa: E731
    for more in (dict(mask=plan), dict(docs=ids), dict(docs=(ids, ids))):
        O = layer(qkv, lambda q, k, v: fa.attention(q, k, v.contiguous(), True, softcap=20.0, slopes=alibi(Hq), **more),
                  turn)
        grad, = torch.autograd.grad(O, qkv, dO)
        # the rotated Q and K are rounded to bf16 on the way (2^-8 of a score's terms): rel-L2 1e-2 covers both
        assert_close("O", O, Or.detach().cpu().numpy(), magnitude=True)
        assert_close("d qkv", grad, gr.cpu().numpy(), magnitude=True)


@gpu
def test_graph_replays_plan_and_both_directions():
    B, H, T, d = 1, 4, 400, 128
    Q, K, V, dO = inputs(B, H, 2, T, T, d, d, seed=14)
    ids, slopes = packed(B, T, 1), alibi(H)

    def step():
        mask = fa.fa_mask_plan(B, T, T, True, 0, ids, ids)
        O, L = fa.fa_forward(Q, K, V, True, softcap=30.0, slopes=slopes, mask=mask)
        return (O, L) + fa.fa_backward(Q, K, V, O, dO, L, True, softcap=30.0, slopes=slopes, mask=mask)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs of the same calls share nothing
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for seed in (2, 3):
        ids.copy_(packed(B, T, seed))
        Q.copy_(inputs(B, H, 2, T, T, d, d, seed=seed)[0])
        want = step()
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
            for a, b in zip(out[2:], want[2:]):  # fp32 sums of dQ meet in any order: one bf16 step
                assert_close("replayed", a, b.double().cpu().numpy(), rel_l2=2.0 ** -8)


@gpu
def test_other_stream():
    B, H, T, d = 1, 4, 700, 64
    Q, K, V, dO = inputs(B, H, 4, T, T, d, d, seed=15)
    ids = packed(B, T, 1)
    want = compare(Q, K, V, dO, True, docs=(ids, ids))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mask = fa.fa_mask_plan(B, T, T, True, 0, ids, ids, stream=s)
    O, L = fa.fa_forward(Q, K, V, True, stream=s, mask=mask)
    dQ, dK, dV = fa.fa_backward(Q, K, V, O, dO, L, True, stream=s, mask=mask)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(O, want[0]) and torch.equal(L, want[1]) and torch.equal(dK, want[3]) and torch.equal(dV, want[4])


@pytest.mark.gpu
def test_no_cap_by_none():
    Q, K, V, _ = inputs(1, 4, 2, 70, 70, 64, 64, 3)
    for got, want in zip(fa.fa_forward(Q, K, V, True, softcap=None, slopes=alibi(4)),
                         fa.fa_forward(Q, K, V, True, slopes=alibi(4))):
        assert torch.equal(got, want)


@gpu
def test_calls_in_a_row_share_plan_results_and_workspace():
    """Kernels that start while the one before them ends must neither read nor
    overwrite early: two batches' steps take turns in the same plan, L, workspace
    and gradient buffers without a wait between them."""
    B, H, Hkv, T, d = 2, 8, 2, 1000, 128
    lib, stream = fa.load(), torch.cuda.current_stream().cuda_stream
    dims = fa.make_dims(B, H, Hkv, T, T, d, d, True, None)
    plan = fa.fa_mask_plan(B, T, T, True, 0, packed(B, T, 1), packed(B, T, 1))
    scores = fa.FaScores(40.0, None, plan.buffer.data_ptr())
    ref = ctypes.byref(dims)
    L = torch.empty(B, H, T, device="cuda")
    ws = torch.empty(lib.fa_backward_scored_workspace_bytes(ref, scores), dtype=torch.uint8, device="cuda")
    batches = []
    for seed in (1, 2):
        Q, K, V, dO = inputs(B, H, Hkv, T, T, d, d, seed=seed)
        batches.append((Q, K, V, dO, packed(B, T, seed + 10), torch.empty_like(Q), [torch.empty_like(t) for t in (Q, K, V)]))

    def step(Q, K, V, dO, ids, O, grads):
        assert lib.fa_mask_plan(ref, ids.data_ptr(), ids.data_ptr(), None, 0, plan.buffer.data_ptr(),
                                plan.buffer.numel() * 4, stream) == fa.FA_OK
        fa.fa_forward(Q, K, V, True, O=O, L=L, softcap=40.0, mask=plan)
        fa.fa_backward(Q, K, V, O, dO, L, True, None, *grads, workspace=ws, softcap=40.0, mask=plan)

    want = []
    for b in batches:
        step(*b)
        torch.cuda.synchronize()
        want.append([b[5].clone()] + [g.clone() for g in b[6]])
        b[5].zero_()
    for turn in range(30):
        for b in batches:
            step(*b)
    torch.cuda.synchronize()
    for b, (O, *grads) in zip(batches, want):
        assert torch.equal(b[5], O)
        for got, g in zip(b[6], grads):  # fp32 sums meet in any order: one bf16 step
            assert_close("in a row", got, g.double().cpu().numpy(), rel_l2=2.0 ** -8)


@gpu
def test_two_streams_at_once():
    B, H, Hkv, T, d = 1, 8, 2, 900, 64
    sets = [inputs(B, H, Hkv, T, T, d, d, seed=s) + (packed(B, T, s),) for s in (31, 32)]

    def step(Q, K, V, dO, ids):
        mask = fa.fa_mask_plan(B, T, T, True, 0, ids, ids)
        O, L = fa.fa_forward(Q, K, V, True, softcap=20.0, slopes=alibi(H), mask=mask)
        return (O, L) + fa.fa_backward(Q, K, V, O, dO, L, True, softcap=20.0, slopes=alibi(H), mask=mask)

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [None, None]
    for turn in range(10):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] = step(*sets[k])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
        for a, b in zip(g[2:], w[2:]):
            assert_close("two streams", a, b.double().cpu().numpy(), rel_l2=2.0 ** -8)


@gpu
def test_offsets_past_32_bits():
    """40 * 8 * 65536 * 128 elements are more than 2^31: the last batch entry's results are those of a call on it
    alone (a window keeps the work small).  dQ is added up in fp32 in any order: one bf16 step."""
    B, H, T, d, W = 40, 8, 65536, 128, 70
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB")
    g = torch.Generator("cuda").manual_seed(4)
    Q, K, V, dO = (torch.empty(B, H, T, d, device="cuda", dtype=bf) for _ in range(4))
    for t in (Q, K, V, dO):
        for b in range(B):
            t[b].copy_(torch.randn(H, T, d, device="cuda", generator=g))
    ids = (torch.arange(T, device="cuda") // 1000).int().expand(B, T).contiguous()
    kw = dict(window=W, softcap=25.0, slopes=alibi(H))
    mask = fa.fa_mask_plan(B, T, T, True, W, ids, ids)
    O, L = fa.fa_forward(Q, K, V, True, mask=mask, **kw)
    grads = fa.fa_backward(Q, K, V, O, dO, L, True, mask=mask, **kw)
    one = [t[B - 1:].contiguous() for t in (Q, K, V, dO)]
    mask1 = fa.fa_mask_plan(1, T, T, True, W, ids[:1], ids[:1])
    O1, L1 = fa.fa_forward(*one[:3], True, mask=mask1, **kw)
    grads1 = fa.fa_backward(*one[:3], O1, one[3], L1, True, mask=mask1, **kw)
    assert torch.equal(O[B - 1:], O1) and torch.equal(L[B - 1:], L1)
    for a, b in zip(grads, grads1):
        off = (a[B - 1:].float() - b.float()).norm() / b.float().norm()
        assert float(off) <= 2.0 ** -8
