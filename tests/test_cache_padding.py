"""Padding rows of fa_cache_attention (those before a sequence's start) see nothing, whatever
their query holds: an empty slot of a batch has what the model made of nothing."""
import math

import pytest
import torch

import tiled_attention_05_gb300 as fa
from test_cache import Setup, check, query


@pytest.mark.gpu
@pytest.mark.parametrize("fill", [math.inf, -math.inf, math.nan, 3.38e38])
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("copies, Hq, Hkv", [(1, 2, 2), (7, 4, 1)])  # a prefix of few rows, and of many
def test_a_padding_row_may_hold_any_query(copies, Hq, Hkv, quant, fill):
    s = Setup([5, 0, 2, 9] * copies, Hkv, 64, 128, quant, 16, [300])
    Q = query(s, Hq, 3)
    for b, n in enumerate(s.lens):
        Q[b, :, :max(3 - n, 0)] = 0
        Q[b, :, :max(3 - n, 0), 0] = fill  # (one channel: scores of both signs and no NaN but the fill's)
    for mods in (dict(), dict(softcap=5.0), dict(window=310)):
        check(s, Q, *fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, **mods), **mods)
    check_alone(s, Q)


def check_alone(s, Q):
    """The same rows without the prefix."""
    s.p_lens = []
    check(s, Q, *fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths))
