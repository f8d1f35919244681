"""The order in which the planned backward takes its key tiles: one super-batch for few
(batch, kv head) groups, the plain rule's super-batches for many, whose live data would not
stay in L2 together; and the parts that they run in where there are few, as many as the
plan leaves work for.  The results are the definition's either way."""
import os
import shutil
import subprocess

import pytest
import torch

import tiled_attention_05_gb300 as fa
from tests.test_scored_attention import alibi, compare, inputs, packed

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tiled_attention_05_gb300", "csrc")
CUDA_INC = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")

PROGRAM = r"""
#include <cstdio>
#include "fa_internal.h"
int main() {
  for (int kv : {1, 16, 32, 64, 256})
    for (int g = 1; g <= 130; ++g)
      std::printf("%d %d %d %d\n", g, kv, fa::planned_super_batch_groups(g, kv, 152), fa::super_batch_groups(g, kv, 152));
  return 0;
}
"""


def test_many_groups_are_not_one_super_batch(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA_INC, "cuda.h")):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "rule.cpp", tmp_path / "rule"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", f"-I{CUDA_INC}", str(src), "-o", str(exe)], check=True)
    table = {}
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        g, kv, planned, plain = map(int, line.split())
        assert g % planned == 0 and planned == (g if g <= 8 else plain)
        table[g, kv] = planned
    assert table[8, 64] == 8     # B 1, 8 kv heads, T 8192
    assert table[64, 64] == 4    # B 8: 256 key tiles at a time, not 4096
    assert table[128, 16] == 16  # B 16, T 2048


@pytest.mark.gpu
@pytest.mark.parametrize("B, Hq, Hkv, T, d, dv, causal", [
    (3, 8, 4, 3500, 64, 64, True),      # 12 groups of 28 key tiles: super-batches
    (7, 4, 2, 3300, 128, 128, False),   # 14 groups, divisors 1, 2, 7, 14
    (1, 6, 3, 13500, 64, 128, True),    # 3 groups of 106: one super-batch
])
def test_planned_backward_in_super_batches(B, Hq, Hkv, T, d, dv, causal):
    ids = packed(B, T, 21)
    Q, K, V, dO = inputs(B, Hq, Hkv, T, T, d, dv, seed=T)
    mods = dict(softcap=30.0, slopes=alibi(Hq), mask=fa.fa_mask_plan(B, T, T, causal, 0, ids, ids))
    O, L = fa.fa_forward(Q, K, V, causal, **mods)
    grads = fa.fa_backward(Q, K, V, O, dO, L, causal, **mods)
    G = Hq // Hkv
    # (some groups by themselves: the score matrices of all are large)
    for b, hk in ((0, 0), (B - 1, Hkv - 1), (B // 2, Hkv // 2)):
        h = slice(hk * G, (hk + 1) * G)
        one = [t[b:b + 1, s].contiguous() for t, s in ((Q, h), (K, slice(hk, hk + 1)), (V, slice(hk, hk + 1)), (dO, h))]
        ids1 = ids[b:b + 1].contiguous()
        # the call on this part alone meets the definition, and is the same up to the order of fp32 sums
        O1, L1, *grads1 = compare(*one, causal, softcap=30.0, slopes=alibi(Hq)[h].contiguous(), docs=(ids1, ids1))
        part = L[b:b + 1, h]
        assert float(torch.where(part == L1, 0.0, (part - L1).abs()).max()) <= 1e-4  # (-inf in both: padding)
        for got, want, s in zip((O, *grads), (O1, *grads1), (h, h, slice(hk, hk + 1), slice(hk, hk + 1))):
            off = (got[b:b + 1, s].float() - want.float()).norm() / want.float().norm()
            assert float(off) <= 2.0 ** -7, float(off)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["short", "one", "a long one among short ones", "prefix"])
@pytest.mark.parametrize("B, Hq, Hkv, T, d, dv", [(1, 8, 2, 1900, 128, 64), (1, 16, 1, 1300, 64, 128), (2, 8, 4, 1000, 64, 64)])
def test_planned_items_in_as_many_parts_as_they_have_work_for(B, Hq, Hkv, T, d, dv, kind):
    """Of 15, 11 and 64 key tiles: some whole, some in two parts, some in up to eight, in one launch."""
    t = torch.arange(T, device="cuda")
    ids = {"short": t // 70, "one": t * 0, "a long one among short ones": torch.where((t > 400) & (t < T - 300), 400, t // 50)}
    Q, K, V, dO = inputs(B, Hq, Hkv, T, T, d, dv, seed=T + len(kind))
    docs = prefix = None
    if kind == "prefix":
        prefix = torch.tensor([T - 100, 30][:B], dtype=torch.int32, device="cuda")
    else:
        ids = ids[kind].int().expand(B, T).contiguous()
        docs = (ids, ids)
    first = compare(Q, K, V, dO, True, softcap=30.0, docs=docs, prefix=prefix, tag=kind)
    again = compare(Q, K, V, dO, True, softcap=30.0, docs=docs, prefix=prefix, tag=kind)
    for a, b in zip(first[3:], again[3:]):  # dK, dV: the parts are added in their order
        assert torch.equal(a, b)
    if docs:
        compare(Q, K, V, dO, False, softcap=30.0, slopes=alibi(Hq), docs=docs, tag=kind + " both ways")
