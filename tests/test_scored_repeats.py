"""Results of the score-modified backward from one call to the next.

Where there are few key tiles, each runs in parts whose fp32 sums of dK and dV the
part that finishes last adds up: always in the parts' order, so that dK and dV are the
same bits every time (as they are where nothing is split, or in two).  dQ is added up
in global memory in any order."""
import pytest
import torch

import tiled_attention_05_gb300 as fa
from tests.test_scored_attention import alibi, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B, Hq, Hkv, T, d, dv, causal", [
    (1, 8, 1, 2048, 128, 128, True),    # 16 key tiles in 8 parts
    (1, 16, 2, 1500, 64, 128, True),
    (1, 32, 1, 640, 128, 64, False),    # 5 key tiles
    (2, 16, 4, 2001, 64, 64, True),     # 2 parts
])
def test_dk_and_dv_are_the_same_every_time(B, Hq, Hkv, T, d, dv, causal):
    Q, K, V, dO = inputs(B, Hq, Hkv, T, T, d, dv, seed=T)
    mods = dict(softcap=30.0, slopes=alibi(Hq))
    O, L = fa.fa_forward(Q, K, V, causal, **mods)
    _, dK, dV = fa.fa_backward(Q, K, V, O, dO, L, causal, **mods)
    for _ in range(30):
        _, dK2, dV2 = fa.fa_backward(Q, K, V, O, dO, L, causal, **mods)
        assert torch.equal(dK2, dK) and torch.equal(dV2, dV)
