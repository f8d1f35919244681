"""Rotary positions of Q and K against the definition in float64, and the
refusals of bad arguments.

Tolerance.  The kernel's cos and sin come from an fp32 argument of at most one
half turn (off by 2^-25 half turns = pi 2^-25 radians) and sincospif (2 ulp),
and two fp32 products and a sum follow: together less than 2^-20 (|x| + |y|)
for the pair (x, y).  The result is rounded once to bf16: half a step, 2^-8 of
the value."""
import ctypes

import pytest
import torch

import tiled_attention_05_gb300 as fa

bf = torch.bfloat16


def reference(x, positions, inv_freq, sections, interleaved, inverse=False):
    """float64 result and the fp32 arithmetic's share of the tolerance."""
    B, H, T, d = x.shape
    n = inv_freq.numel()
    axis = [a for a, k in enumerate(sections) for _ in range(k)]
    pos = positions.to(torch.float64).reshape(len(sections), -1, T).expand(-1, B, -1)
    # whole turns leave before the product: positions and 2 pi meet in long integers' range exactly
    theta = torch.stack([pos[a] * inv_freq[f].double() for f, a in enumerate(axis)], -1) if n else pos.new_zeros(B, T, 0)
    theta = -theta if inverse else theta
    c, s = theta.cos()[:, None], theta.sin()[:, None]
    y, slack = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., i].double(), x[..., j].double()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    slack[..., i] = slack[..., j] = 2.0 ** -20 * (a.abs() + b.abs())
    return y, slack


def check(got, x, positions, inv_freq, sections, interleaved, inverse=False):
    y, slack = reference(x, positions, inv_freq, sections, interleaved, inverse)
    off = (got.double() - y).abs() - (slack + 2.0 ** -8 * y.abs())
    assert off.numel() == 0 or float(off.max()) <= 0, float(off.max())


def freqs(n, base=1e6, device="cuda"):
    return (base ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))).float().to(device)


# ---------------------------------------------------------------- refusals (CPU)
def cpu_call(**kw):
    a = dict(Q=torch.zeros(1, 4, 8, 64, dtype=bf), K=torch.zeros(1, 2, 8, 64, dtype=bf),
             positions=torch.zeros(1, 1, 8, dtype=torch.int32), inv_freq=torch.zeros(32))
    a.update(kw)
    return fa.fa_rotary(**a)


@pytest.mark.parametrize("bad, why", [
    (dict(), "CUDA"),
    (dict(Q=torch.zeros(4, 8, 64, dtype=bf)), "B, H, T, d"),
    (dict(inv_freq=torch.zeros(33)), "inv_freq has shape"),
    (dict(inv_freq=torch.zeros(2, 16)), "inv_freq has shape"),
    (dict(sections=[16, 15]), "add up"),
    (dict(sections=[40, -8]), "add up"),
    (dict(sections=[8, 8, 8, 4, 4]), "one to four"),
])
def test_refuses(bad, why):
    with pytest.raises(ValueError, match=why):
        cpu_call(**bad)


def dims(**kw):
    z = dict(B=1, Hq=4, Hk=2, T=8, d=64, rot=64, axes=1, interleaved=0, pos_bytes=4, section=(32, 0, 0, 0),
             q_stride=(2048, 512, 64))
    z.update(kw)
    s3, qs = ctypes.c_longlong * 3, z["q_stride"]
    return fa.FaRotaryDims(*(z[k] for k in ("B", "Hq", "Hk", "T", "d", "rot", "axes", "interleaved", "pos_bytes")),
                           (ctypes.c_int * 4)(*z["section"]), s3(*qs), s3(1024, 512, 64), s3(2048, 512, 64),
                           s3(1024, 512, 64), 8, 8)


def abi_call(d, ptrs=(0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000), inverse=0):
    q, k, pos, f, qo, ko = ptrs
    return fa.load().fa_rotary(ctypes.byref(d), q, k, pos, f, qo, ko, inverse, None)


@pytest.mark.parametrize("bad", [dict(B=-1), dict(T=-1), dict(Hk=-1), dict(rot=80), dict(rot=-16), dict(axes=0), dict(axes=5),
                                 dict(interleaved=2), dict(pos_bytes=2), dict(section=(31, 0, 0, 0)),
                                 dict(axes=2, section=(40, -8, 0, 0)), dict(q_stride=(2048, 512, 60))])
def test_abi_refuses_bad_dims(bad):
    assert abi_call(dims(**bad)) == fa.FA_ERR_INVALID_ARG


def test_abi_refuses_the_rest():
    assert fa.load().fa_rotary(None, 0, 0, 0, 0, 0, 0, 0, None) == fa.FA_ERR_INVALID_ARG
    assert abi_call(dims(), inverse=2) == fa.FA_ERR_INVALID_ARG
    for bad in ((0, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000), (0x1008, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000),
                (0x1000, 0x2000, 0, 0x4000, 0x5000, 0x6000), (0x1000, 0x2000, 0x3002, 0x4000, 0x5000, 0x6000),
                (0x1000, 0x2000, 0x3000, 0x4001, 0x5000, 0x6000), (0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6008)):
        assert abi_call(dims(), bad) == fa.FA_ERR_INVALID_ARG
    assert abi_call(dims(d=96, rot=64)) == fa.FA_ERR_UNSUPPORTED
    assert abi_call(dims(rot=24, section=(12, 0, 0, 0))) == fa.FA_ERR_UNSUPPORTED
    assert abi_call(dims(Hq=60000, Hk=6000)) == fa.FA_ERR_UNSUPPORTED
    assert abi_call(dims(T=0), (0,) * 6) == fa.FA_OK
    assert abi_call(dims(Hq=0, Hk=0), (0,) * 6) == fa.FA_OK


# ---------------------------------------------------------------- parity (GPU)
CASES = [
    # B, Hq, Hk, T, d, sections, interleaved, first position
    (1, 1, 1, 1, 64, (32,), False, 0),
    (2, 3, 1, 5, 64, (16,), False, 7),             # half of the channels turned
    (3, 4, 2, 37, 128, (16, 24, 24), False, 100000),
    (2, 6, 2, 33, 128, (32, 0, 16), True, -50),     # an axis without frequencies; a quarter copied; behind the start
    (1, 9, 1, 130, 64, (2, 3, 1, 2), True, 3),      # four axes, odd sections, heads not a multiple of four
    (1, 32, 8, 700, 128, (64,), False, 2 ** 30),    # far positions
    (40, 2, 2, 1, 128, (20, 44), False, 12345),     # one token of many requests
    (1, 2, 0, 6, 64, (32,), False, 0),             # no K
    (1, 1, 1, 9, 128, (), False, 0),               # nothing turned: a copy
]


@pytest.mark.gpu
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:5])))
def test_parity(case, inverse):
    B, Hq, Hk, T, d, sections, inter, first = case
    g = torch.Generator("cuda").manual_seed(sum(case[:5]))
    sections = sections or (0,)
    Q, K = (torch.randn(B, H, T, d, generator=g, device="cuda").to(bf) for H in (Hq, Hk))
    pos = first + torch.randint(0, 999, (len(sections), B, T), generator=g, device="cuda", dtype=torch.int32)
    f = freqs(sum(sections))
    call = fa.fa_rotary_backward if inverse else fa.fa_rotary
    for p in (pos, pos.long()):
        Qr, Kr = call(Q, K, p, f, sections=sections, interleaved=inter)
        for got, x in ((Qr, Q), (Kr, K)):
            check(got, x, pos, f, sections, inter, inverse)
            assert torch.equal(got[..., 2 * sum(sections):], x[..., 2 * sum(sections):])
    # in place
    Qi, Ki = Q.clone(), K.clone()
    call(Qi, Ki, pos, f, sections, inter, Qi, Ki)
    assert torch.equal(Qi, Qr) and torch.equal(Ki, Kr)


@pytest.mark.gpu
def test_packed_projection_and_shared_positions():
    B, T, Hq, Hk, d = 2, 45, 4, 2, 128
    g = torch.Generator("cuda").manual_seed(3)
    qkv = torch.randn(B, T, (Hq + 2 * Hk) * d, generator=g, device="cuda").to(bf).view(B, T, Hq + 2 * Hk, d)
    Q, K = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hk].transpose(1, 2)
    f, pos = freqs(64), torch.arange(T, device="cuda", dtype=torch.int32) + 500
    want = fa.fa_rotary(Q.contiguous(), K.contiguous(), pos.expand(1, B, T).contiguous(), f)
    for p in (pos, pos.expand(B, T), pos.expand(1, B, T), torch.stack((pos, pos), 1)[:, 0]):
        got = fa.fa_rotary(Q, K, p, f)
        assert got[0].is_contiguous() and all(torch.equal(a, b) for a, b in zip(got, want))
    check(want[0], Q, pos.expand(1, B, T), f, (64,), False)
    two = torch.stack((pos, pos * 2))                       # [axes, T]
    got = fa.fa_rotary(Q, K, two, f, sections=(40, 24))
    check(got[1], K, two[:, None].expand(2, B, T), f, (40, 24), False)
    for bad in (Q[..., 1:65], Q[..., ::2], torch.zeros(B, Hq, T, d + 4, device="cuda", dtype=bf)[..., :d]):
        with pytest.raises(ValueError, match="strides"):
            fa.fa_rotary(bad, torch.zeros(B, Hk, T, bad.shape[3], device="cuda", dtype=bf), pos, f[:16])
    with pytest.raises(ValueError, match="positions has shape"):
        fa.fa_rotary(Q, K, pos[1:], f)
    with pytest.raises(ValueError, match="int32 or int64"):
        fa.fa_rotary(Q, K, pos.float(), f)


@pytest.mark.gpu
def test_frequencies_of_any_size_and_sign():
    B, H, T, d = 1, 2, 64, 64
    g = torch.Generator("cuda").manual_seed(4)
    Q = torch.randn(B, H, T, d, generator=g, device="cuda").to(bf)
    f = torch.tensor([1.0, -1.0, 3.5, -0.37, 6.2831855, 1e-30, 0.0, 2e-39] * 4, device="cuda")
    pos = torch.randint(-99, 100, (1, 1, T), generator=g, device="cuda", dtype=torch.int64)
    check(fa.fa_rotary(Q, Q, pos, f)[0], Q, pos, f, (32,), False)
    far = torch.full((1, 1, T), -(2 ** 62) // 3, device="cuda", dtype=torch.int64)
    once = fa.fa_rotary(Q, Q, far, f)[0]
    back = fa.fa_rotary_backward(once, once, far, f)[0]
    # two rotations, each rounded: 2^-8 of the pair's length and of the result
    pair = (Q.double()[..., :32].square() + Q.double()[..., 32:].square()).sqrt().repeat(1, 1, 1, 2)
    assert bool(((back.double() - Q.double()).abs() <= 2.0 ** -7 * 1.5 * pair + 2.0 ** -8 * Q.double().abs()).all())


@pytest.mark.gpu
def test_gradient_is_the_transposed_map_and_flows_to_the_projection():
    B, T, Hq, Hk, d = 2, 19, 4, 2, 64
    g = torch.Generator("cuda").manual_seed(5)
    qkv = torch.randn(B, T, Hq + Hk, d, generator=g, device="cuda").to(bf).requires_grad_()
    pos = torch.randint(0, 5000, (2, B, T), generator=g, device="cuda", dtype=torch.int32)
    f = freqs(24)
    Q, K = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:].transpose(1, 2)
    Qr, Kr = fa.rotary(Q, K, pos, f, (10, 14))
    dQr, dKr = (torch.randn(x.shape, generator=g, device="cuda").to(bf) for x in (Qr, Kr))
    grad, = torch.autograd.grad((Qr, Kr), qkv, (dQr, dKr))
    check(grad[:, :, :Hq].transpose(1, 2), dQr, pos, f, (10, 14), False, inverse=True)
    check(grad[:, :, Hq:].transpose(1, 2), dKr, pos, f, (10, 14), False, inverse=True)
    # an expanded gradient (stride 0) is taken too
    Qr, Kr = fa.rotary(Q, K, pos, f, (10, 14))
    a, = torch.autograd.grad(Qr.sum(), qkv)
    check(a[:, :, :Hq].transpose(1, 2), torch.ones_like(Qr), pos, f, (10, 14), False, inverse=True)
    with pytest.raises(ValueError, match="no gradient"):
        fa.rotary(Q, K, pos, f.clone().requires_grad_(), (10, 14))


@pytest.mark.gpu
def test_other_stream_and_graph():
    B, H, T, d = 1, 4, 300, 128
    g = torch.Generator("cuda").manual_seed(6)
    Q = torch.randn(B, H, T, d, generator=g, device="cuda").to(bf)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    f = freqs(64)
    want = fa.fa_rotary(Q, Q, pos, f)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fa.fa_rotary(Q, Q, pos, f, stream=s)[0]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.fa_rotary(Q, Q, pos, f)[0]
    pos.add_(11)
    graph.replay()
    torch.cuda.synchronize()
    check(out, Q, pos.view(1, 1, T), f, (64,), False)


@pytest.mark.gpu
def test_gradient_of_the_gradient():
    """The rotation is linear: the gradient (R^T g) has the gradient R u in g, by the same kernels exactly."""
    B, Hq, Hk, T, d, sections = 2, 3, 1, 21, 64, (8, 12, 12)
    g = torch.Generator("cuda").manual_seed(5)
    Q, K, gq, gk = (torch.randn(B, H, T, d, device="cuda", dtype=bf, generator=g).requires_grad_() for H in (Hq, Hk, Hq, Hk))
    pos = torch.randint(0, 5000, (3, B, T), device="cuda", dtype=torch.int32, generator=g)
    f = freqs(32)
    Qr, Kr = fa.rotary(Q, K, pos, f, sections)
    dQ, dK = torch.autograd.grad((Qr, Kr), (Q, K), (gq, gk), create_graph=True)
    for got, want in zip((dQ, dK), fa.fa_rotary_backward(gq.detach(), gk.detach(), pos, f, sections)):
        assert torch.equal(got, want)
    uq, uk = torch.randn_like(dQ), torch.randn_like(dK)
    ddq, ddk = torch.autograd.grad((dQ, dK), (gq, gk), (uq, uk))
    for got, want in zip((ddq, ddk), fa.fa_rotary(uq, uk, pos, f, sections)):
        assert torch.equal(got, want)


@pytest.mark.gpu
def test_turns_in_a_row_in_place():
    """Turned in place forth and back, with no wait in between: each call reads what the one before it wrote."""
    B, H, T, d = 2, 4, 1200, 64
    g = torch.Generator("cuda").manual_seed(9)
    Q, K = (torch.randn(B, H, T, d, device="cuda", dtype=bf, generator=g) for _ in range(2))
    pos, f = torch.arange(T, device="cuda", dtype=torch.int32), freqs(32)
    want_q, want_k = Q.clone(), K.clone()
    for _ in range(20):
        fa.fa_rotary(Q, K, pos, f, Qo=Q, Ko=K)
        fa.fa_rotary_backward(Q, K, pos, f, dQ=Q, dK=K)
        torch.cuda.synchronize()
    for _ in range(20):
        fa.fa_rotary(want_q, want_k, pos, f, Qo=want_q, Ko=want_k)
        fa.fa_rotary_backward(want_q, want_k, pos, f, dQ=want_q, dK=want_k)
    assert torch.equal(Q, want_q) and torch.equal(K, want_k)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Three rows of 2^23 tokens are 3 * 2^30 elements in and out: the last row is that of a call on it alone."""
    B, T, d = 3, 1 << 23, 128
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.empty(B, T, 1, d, device="cuda", dtype=bf)
    x.view(-1, 1 << 20).copy_(torch.randn(1 << 20, device="cuda", generator=torch.Generator("cuda").manual_seed(3)))
    x = x.transpose(1, 2)
    none = torch.empty(B, 0, T, d, device="cuda", dtype=bf)
    pos, f = torch.arange(B * T, device="cuda", dtype=torch.int64).view(1, B, T), freqs(64)
    y, _ = fa.fa_rotary(x, none, pos, f)
    one, _ = fa.fa_rotary(x[2:], none[2:], pos[:, 2:], f)
    assert torch.equal(y[2:], one)
    tail = slice(T - 64, T)
    check(one[:, :, tail], x[2:, :, tail], pos[:, 2:, tail], f, (64,), False)
