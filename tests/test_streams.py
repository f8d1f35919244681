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
