"""Calls with an explicit stream, with the current stream busy meanwhile: what a call
makes for itself (copies, scratch, results) is ordered with the stream it runs on."""
import pytest
import torch

import tiled_attention_05_gb300 as fa

bf = torch.bfloat16


@pytest.fixture(scope="module")
def busy():
    """Some milliseconds of work on the current stream (in buffers of its own)."""
    a = torch.ones(8192, 8192, device="cuda", dtype=bf)
    out = torch.empty_like(a)

    def work(n=12):
        for _ in range(n):
            torch.matmul(a, a, out=out)

    work(1)
    torch.cuda.synchronize()
    return work


@pytest.mark.gpu
@pytest.mark.parametrize("call", [fa.fa_rotary, fa.fa_rotary_backward])
def test_positions_that_have_to_be_copied(call, busy):
    B, H, T, d = 2, 4, 3000, 64
    g = torch.Generator("cuda").manual_seed(1)
    Q, K = (torch.randn(B, H, T, d, device="cuda", generator=g).to(bf) for _ in range(2))
    pos = torch.randint(0, 5000, (B, T, 3), device="cuda", dtype=torch.int32, generator=g)
    strided = pos.permute(2, 0, 1)  # [axes, B, T], tokens not next to each other
    f = (1e4 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    want = call(Q, K, strided.contiguous(), f, (10, 12, 10))
    torch.cuda.synchronize()
    s, got = torch.cuda.Stream(), [torch.empty_like(t) for t in (Q, K)]
    for _ in range(5):
        poison = torch.full((3, B, T), 77, device="cuda", dtype=torch.int32)
        del poison  # what an unordered copy would find in its place
        s.wait_stream(torch.cuda.current_stream())
        busy()  # after the wait: the other stream does not wait for its end
        call(Q, K, strided, f, (10, 12, 10), False, *got, stream=s)
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        torch.cuda.synchronize()


def step(Q, K, V, dO, slopes, ids, stream=None):
    """A plan, a forward that is split over the keys and a backward in parts."""
    B, T = ids.shape
    mask = fa.fa_mask_plan(B, T, T, True, 0, ids, ids, stream=stream)
    mods = dict(softcap=30.0, slopes=slopes, mask=mask, stream=stream)
    O, L = fa.fa_forward(Q, K, V, True, **mods)
    return (O, L) + fa.fa_backward(Q, K, V, O, dO, L, True, **mods)


def batches(B, Hq, Hkv, T, d, seeds):
    out = []
    for seed in seeds:
        g = torch.Generator("cuda").manual_seed(seed)
        Q, K, V, dO = (torch.randn(B, H, T, d, device="cuda", generator=g).to(bf) for H in (Hq, Hkv, Hkv, Hq))
        slopes = (torch.rand(Hq, device="cuda", generator=g) / 16)
        ids = (torch.arange(T, device="cuda") // (T // seed)).int().expand(B, T).contiguous()
        out.append((Q, K, V, dO, slopes, ids))
    return out


def same(got, want):
    """The first two (O, L) and what is not a gradient are the same bits; dQ, dK and dV are added up in fp32, in an
    order of their own, and rounded once (2^-8)."""
    for n, (a, b) in enumerate(zip(got, want)):
        if 2 <= n < 5:
            assert float((a.float() - b.float()).norm()) <= 2.0 ** -8 * float(b.float().norm()), n
        else:
            assert torch.equal(a, b), n


@pytest.mark.gpu
def test_current_and_explicit_stream_in_turn():
    """No call waits for the other stream's: scratch and results must not be shared between them."""
    sets = batches(1, 4, 2, 2048, 64, (2, 3))
    want = [[t.clone() for t in step(*b)] for b in sets]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(10):
        got = []
        for _ in range(5):
            got.append((step(*sets[0]), step(*sets[1], stream=s)))
        torch.cuda.synchronize()
        for here, there in got:
            same(here, want[0])
            same(there, want[1])


@pytest.mark.gpu
def test_memory_freed_while_the_current_stream_still_uses_it(busy):
    """Blocks freed here, with their last use still queued here, are not what a call on another stream writes to."""
    (Q, K, V, dO, slopes, ids), = batches(1, 4, 2, 1024, 64, (2,))
    g = torch.Generator("cuda").manual_seed(7)
    f, pos = torch.rand(32, device="cuda", generator=g), torch.arange(1024, device="cuda", dtype=torch.int32)
    want = step(Q, K, V, dO, slopes, ids) + fa.fa_rotary(Q, K, pos, f)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        busy()
        late = [torch.full((n,), 9, device="cuda", dtype=torch.uint8) for n in (2 ** 17, 2 ** 19, 2 ** 20, 2 ** 21, 2 ** 22)]
        del late  # written after the work that is queued here
        got = step(Q, K, V, dO, slopes, ids, stream=s) + fa.fa_rotary(Q, K, pos, f, stream=s)
        torch.cuda.synchronize()
        same(got, want)


@pytest.mark.gpu
def test_results_freed_while_the_current_stream_still_reads_them(busy):
    """Results made on another stream and dropped with a read of them queued here are not written by its next call."""
    sets = batches(1, 4, 2, 1024, 64, (2, 3))
    want = fa.fa_forward(*sets[0][:3], True)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        O, _ = fa.fa_forward(*sets[0][:3], True, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        busy()
        copy = O.clone()
        del O
        for _ in range(3):
            fa.fa_forward(*sets[1][:3], True, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(copy, want)


@pytest.mark.gpu
def test_explicit_stream_inside_a_captured_graph():
    first, other = batches(1, 4, 2, 900, 64, (2, 3))
    static = [t.clone() for t in first]
    step(*static)
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        out = step(*static, stream=s)
        torch.cuda.current_stream().wait_stream(s)
    for b in (other, first):
        for t, new in zip(static, b):
            t.copy_(new)
        want = step(*b)
        graph.replay()
        torch.cuda.synchronize()
        same(out, want)
