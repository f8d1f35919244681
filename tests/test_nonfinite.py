"""NaN and infinity in Q, K and V, and the largest values that a capped call takes.

A NaN in a query row, or in a key that a row sees, makes that row's weights NaN, and
so its O and its L, whether the call is split over its keys or not; other rows are
what they are without it, bit for bit.  A NaN in V reaches the channel it is in, of
every row that sees its key.  (Masked places have to hold finite values.)

Under a cap a score of any size counts as the cap; the tolerances are those of
test_scored_attention: O off by r |O| + sum_j (r + e) P_ij |V_j| with r = 2^-8 and
e = 2^-12 + 2^-20 c, L by 1e-4 + 2^-20 c."""
import ctypes
import math

import pytest
import torch

import tiled_attention_05_gb300 as fa
from tests.test_scored_attention import alibi, definition, inputs, visible

pytestmark = pytest.mark.gpu

NAN = float("nan")
# name, cap, slopes, mask: every form of the scores (a cap of 200 is past the bounded form)
FORMS = [("plain", 0.0, False, False), ("mask", 0.0, False, True), ("cap", 20.0, False, False), ("slopes", 0.0, True, False),
         ("both", 50.0, True, False), ("wide cap", 200.0, True, False), ("capped documents", 30.0, False, True)]
# B, Hq, Hkv, Tq, Tk, d, dv: packed and split, split, one item per head (split by nothing)
SHAPES = [(1, 8, 2, 32, 4000, 128, 128), (1, 8, 8, 2048, 2048, 64, 64), (2, 4, 2, 300, 300, 128, 64)]


def forward(Q, K, V, cap, slopes, mask, workspace):
    """O, L of the causal call, with or without the workspace that lets it split."""
    if workspace:
        return fa.fa_forward(Q, K, V, True, softcap=cap, slopes=slopes, mask=mask)
    B, Hq, Tq, d = Q.shape
    dims = fa.make_dims(B, Hq, K.shape[1], Tq, K.shape[2], d, V.shape[3], True, None)
    scores = fa.FaScores(cap, slopes.data_ptr() if slopes is not None else None,
                         mask.buffer.data_ptr() if mask is not None else None)
    O, L = Q.new_empty(B, Hq, Tq, V.shape[3]), torch.empty(B, Hq, Tq, device=Q.device)
    code = fa.load().fa_forward_scored(ctypes.byref(dims), ctypes.byref(scores), Q.data_ptr(), K.data_ptr(), V.data_ptr(),
                                       O.data_ptr(), L.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
    assert code == fa.FA_OK
    return O, L


def problem(shape, form):
    B, Hq, Hkv, Tq, Tk, d, dv = shape
    _, cap, slopes, masked = form
    Q, K, V, dO = inputs(B, Hq, Hkv, Tq, Tk, d, dv, seed=Tk + d)
    slopes = alibi(Hq) / 64 if slopes else None  # (gentle: no weight of a row of this length underflows)
    mask = None
    if masked:  # one document: rows see what the causal mask shows
        ids = torch.zeros(B, max(Tq, Tk), dtype=torch.int32, device="cuda")
        mask = fa.fa_mask_plan(B, Tq, Tk, True, 0, ids[:, :Tq].contiguous(), ids[:, :Tk].contiguous())
    return Q, K, V, dO, cap, slopes, mask


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: f[0])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_a_nan_reaches_the_rows_that_see_it(shape, form, workspace):
    B, Hq, Hkv, Tq, Tk, d, dv = shape
    Q, K, V, dO, cap, slopes, mask = problem(shape, form)
    O0, L0 = forward(Q, K, V, cap, slopes, mask, workspace)
    assert bool(torch.isfinite(O0).all()) and bool(torch.isfinite(L0).all())
    b, hk, j = B - 1, Hkv - 1, Tk // 3
    heads = slice(hk * (Hq // Hkv), Hq)
    first = max(0, j - (Tk - Tq))  # first row that sees key j
    behind = 128 * (first // 128)  # rows before it in its tile have the NaN at a masked place

    def others(t):
        t = t.clone()
        t[b, heads, behind:] = 0
        return t

    bad = K.clone()
    bad[b, hk, j, 5] = NAN
    O, L = forward(Q, bad, V, cap, slopes, mask, workspace)
    assert bool(O[b, heads, first:].isnan().all()) and bool(L[b, heads, first:].isnan().all())
    assert torch.equal(others(O), others(O0)) and torch.equal(others(L), others(L0))

    bad = V.clone()
    bad[b, hk, j, 7] = NAN
    O, L = forward(Q, K, bad, cap, slopes, mask, workspace)
    assert bool(O[b, heads, first:, 7].isnan().all())
    keep = torch.arange(dv, device="cuda") != 7
    assert torch.equal(O[b, heads, first:][..., keep], O0[b, heads, first:][..., keep]) and torch.equal(L, L0)

    bad = Q.clone()
    h, i = heads.start, Tq - 3
    bad[b, h, i, 1] = NAN
    O, L = forward(bad, K, V, cap, slopes, mask, workspace)
    assert bool(O[b, h, i].isnan().all()) and bool(L[b, h, i].isnan())
    O[b, h, i], L[b, h, i] = O0[b, h, i], L0[b, h, i]
    assert torch.equal(O, O0) and torch.equal(L, L0)


@pytest.mark.parametrize("form", FORMS, ids=lambda f: f[0])
def test_a_nan_reaches_the_gradients(form):
    """A row of NaN weights gives NaN to its dQ and to dK and dV of every key it sees."""
    shape = B, Hq, Hkv, Tq, Tk, d, dv = SHAPES[2]
    Q, K, V, dO, cap, slopes, mask = problem(shape, form)
    i = 140
    Q[0, 1, i, 3] = NAN
    mods = dict(softcap=cap, slopes=slopes, mask=mask)
    O, L = fa.fa_forward(Q, K, V, True, **mods)
    dQ, dK, dV = fa.fa_backward(Q, K, V, O, dO, L, True, **mods)
    assert bool(dQ[0, 1, i].isnan().all())
    assert bool(dK[0, 0, :i + 1].isnan().all()) and bool(dV[0, 0, :i + 1].isnan().all())
    for t in (dQ[1], dK[1], dV[1], dK[0, 1], dV[0, 1], dQ[0, 0]):
        assert bool(torch.isfinite(t).all())
    # a key: every row from it on has NaN weights, and every key is seen by one of them
    Q, K, V, dO, cap, slopes, mask = problem(shape, form)
    K[0, 1, 100, 0] = NAN
    O, L = fa.fa_forward(Q, K, V, True, **mods)
    dQ, dK, dV = fa.fa_backward(Q, K, V, O, dO, L, True, **mods)
    assert bool(dQ[0, 2:, 100:].isnan().all()) and bool(dV[0, 1].isnan().all()) and bool(dK[0, 1].isnan().all())
    for t in (dQ[1], dK[1], dV[1], dK[0, 0], dV[0, 0], dQ[0, :2]):
        assert bool(torch.isfinite(t).all())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cap, slopes", [(5.0, False), (5.0, True), (100.0, True)])
def test_a_nan_row_leaves_the_other_rows_gradients(cap, slopes, causal):
    """dQ of the rows beside a NaN row is what it is without it, also where one reciprocal serves four rows' capped
    scores (past half the cap).  dQ is added up in fp32 in any order and rounded once: 2^-8 of the whole."""
    B, Hq, Hkv, T, d = 1, 4, 2, 300, 64
    Q, K, V, dO = inputs(B, Hq, Hkv, T, T, d, d, seed=5, std=8.0 * cap / 5)
    mods = dict(softcap=cap, slopes=alibi(Hq) if slopes else None)

    def dq(Q):
        O, L = fa.fa_forward(Q, K, V, causal, **mods)
        return fa.fa_backward(Q, K, V, O, dO, L, causal, **mods)[0]

    want = dq(Q)
    bad = Q.clone()
    bad[0, 1, 141, 3] = bad[0, 3, 10, 0] = NAN
    got = dq(bad)
    assert bool(got[0, 1, 141].isnan().all()) and bool(got[0, 3, 10].isnan().all())
    got[0, 1, 141], got[0, 3, 10] = want[0, 1, 141], want[0, 3, 10]
    assert bool(torch.isfinite(got).all())
    assert float((got.float() - want.float()).norm()) <= 2.0 ** -8 * float(want.float().norm())


@pytest.mark.parametrize("cap, slopes", [(20.0, False), (50.0, True), (200.0, True)])
@pytest.mark.parametrize("Tq, Tk", [(32, 4000), (300, 300)])
def test_infinite_scores_count_as_the_cap(Tq, Tk, cap, slopes):
    B, Hq, Hkv, d = 1, 4, 2, 64
    Q, K, V, _ = inputs(B, Hq, Hkv, Tq, Tk, d, d, seed=Tk)
    Q[0, 0, 20], Q[0, 1, 21] = 2.0 ** 100, -2.0 ** 100
    K[0, 0, 9] = 2.0 ** 100  # q.k = +-2^206, past fp32
    slopes = alibi(Hq) if slopes else None
    O, L = fa.fa_forward(Q, K, V, True, softcap=cap, slopes=slopes)
    vis = visible(B, Tq, Tk, True, device="cuda")
    Or, Lr, P, _ = definition(Q.double(), K.double(), V.double(), vis, cap, slopes, more=True)
    r, e = 2.0 ** -8, 2.0 ** -12 + 2.0 ** -20 * cap
    bound = r * Or.abs() + (r + e) * torch.matmul(P, V.double().abs().repeat_interleave(Hq // Hkv, 1))
    assert bool(((O.double() - Or).abs() <= bound).all())
    assert float((L - Lr).abs().max()) <= 1e-4 + 2.0 ** -20 * cap


@pytest.mark.parametrize("cap", [62.0, 60.0, 55.0])
@pytest.mark.parametrize("Tq", [1, 100])
def test_large_values_of_many_capped_keys(cap, Tq):
    """Values just below 2^20 under weights of 2^90, over 2^19 keys: the unnormalised sums stay inside fp32.
    Scores are saturated at both ends, so O is the mean of the values of the keys at the upper one.  Each of the
    sums of O and L (at most 2^12 terms one after the other, of one sign, each addition off by 2^-23 of the sum so far
    at most) is off by 2^-11 of itself; O is rounded once, 2^-8, and P before it, 2^-8."""
    Tk, d = 1 << 19, 64
    g = torch.Generator("cuda").manual_seed(6)
    sign = torch.where(torch.rand(Tk, generator=g, device="cuda") < 0.9, 8.0, -8.0)
    Q = torch.full((1, 1, Tq, d), 8.0, device="cuda").bfloat16()
    K = sign[:, None].expand(Tk, d).bfloat16()[None, None].contiguous()
    V = (2.0 ** 20 * (1 - 2.0 ** -8) * (1 - 0.1 * torch.rand(Tk, d, generator=g, device="cuda"))).bfloat16()[None, None]
    assert float(V.max()) < 2.0 ** 20
    O, L = fa.fa_forward(Q, K, V, False, softcap=cap)
    up = sign > 0
    want = V[0, 0][up].double().mean(0)
    off = (O[0, 0].double() - want).abs() / want
    assert float(off.max()) <= 2 * 2.0 ** -8 + 2 * 2.0 ** -11, float(off.max())
    assert float((L - (cap + math.log(int(up.sum())))).abs().max()) <= 1e-4 + 2.0 ** -20 * cap + 2.0 ** -11
