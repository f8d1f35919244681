"""Keys and values that no row sees, or that some rows do not see, leave no trace in their results."""
import math

import pytest
import torch

import tiled_attention_05_gb300 as fa
from test_cache import Setup, bf, check, query, slopes_of

MANY, FEW = [30] * 20, [30] * 3  # sequences of a group: 80 rows of a kv head, and 12


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [MANY, FEW])
@pytest.mark.parametrize("softcap", [0.0, 1.0, 30.0])
def test_nan_key_beside_the_first_visible_one(lens, softcap):
    """A row with a NaN has a NaN scale in an e4m3 cache.  Where the window hides it, the keys
    beside it keep their scores, whichever of a four of them it is."""
    s = Setup(lens, 1, 64, 64, True, 16, [400])
    Q = query(s, 4, 1, std=2.0)
    K, V = (torch.full((1, 1, 1, 64), x, device="cuda").to(bf) for x in (math.nan, 1.0))
    at = torch.tensor([200], dtype=torch.int32, device="cuda")
    fa.fa_cache_write(s.cache, K, V, s.p_tables, at)
    for first in range(201, 209):  # the first key that is seen
        mods = dict(window=400 + 29 - first + 1, softcap=softcap)
        check(s, Q, *fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, **mods), **mods)
