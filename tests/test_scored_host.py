"""Host side of the score-modified calls."""
import subprocess
import sys
import textwrap

import pytest
import torch

import tiled_attention_05_gb300 as fa


def test_workspace_queries_without_heads():
    """Hq = Hkv = 0 is a problem of size zero.  (In a process of its own: a division by the number of heads ends it.)"""
    code = textwrap.dedent("""
        import ctypes
        import tiled_attention_05_gb300 as fa
        lib, scores = fa.load(), fa.FaScores(5.0, None, None)
        for B, Hq, Hkv in ((1, 0, 0), (1, 0, 2), (0, 4, 2)):
            dims = fa.make_dims(B, Hq, Hkv, 5, 7000, 64, 64, True, None)
            assert lib.fa_forward_scored_workspace_bytes(ctypes.byref(dims), ctypes.byref(scores)) == 0
            lib.fa_backward_scored_workspace_bytes(ctypes.byref(dims), ctypes.byref(scores))
            assert lib.fa_forward_scored(ctypes.byref(dims), ctypes.byref(scores), *[0x1000] * 5, None, 0, None) == fa.FA_OK
        """)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr)


@pytest.mark.gpu
@pytest.mark.parametrize("B, Hq, Hkv", [(1, 0, 0), (1, 0, 2), (0, 4, 2)])
def test_calls_without_heads_or_batch(B, Hq, Hkv):
    Q, K = (torch.zeros(B, H, 9, 64, device="cuda", dtype=torch.bfloat16) for H in (Hq, Hkv))
    slopes = torch.zeros(Hq, device="cuda")
    O, L = fa.fa_forward(Q, K, K, True, softcap=5.0, slopes=slopes)
    dQ, dK, dV = fa.fa_backward(Q, K, K, O, O, L, True, softcap=5.0, slopes=slopes)
    torch.cuda.synchronize()
    assert O.shape == Q.shape and L.shape == (B, Hq, 9) and dQ.shape == Q.shape
    assert not dK.any() and not dV.any()


def test_a_gradient_of_the_gradient_is_refused(monkeypatch):
    """The backward kernels have no gradient: a gradient penalty through attention raises, and does not lose its term.
    (On the CPU, with the two calls replaced by sums that have one.)"""
    monkeypatch.setattr(fa, "fa_forward", lambda Q, K, V, *a, **kw: (Q * K + V, Q.sum(-1)))
    monkeypatch.setattr(fa, "fa_backward", lambda Q, K, V, O, dO, L, *a, **kw: (dO * K, dO * Q, dO * 1))
    Q, K, V = (torch.randn(1, 2, 3, 4, requires_grad=True) for _ in range(3))
    O = fa.attention(Q, K, V, softcap=20.0)
    dQ, = torch.autograd.grad(O.sum(), Q, create_graph=True)
    assert torch.equal(dQ, K)
    with pytest.raises(RuntimeError, match="differentiated again"):
        (O.sum() + dQ.square().sum()).backward()
    w = torch.randn_like(O).requires_grad_()  # also through the gradient that comes in
    dV, = torch.autograd.grad((w * fa.attention(Q, K, V)).sum(), V, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated again"):
        dV.square().sum().backward()
    fa.attention(Q, K, V, softcap=20.0).sum().backward()  # the first gradient is what it was
    assert torch.equal(Q.grad, K) and torch.equal(K.grad, Q) and torch.equal(V.grad, torch.ones_like(V))
