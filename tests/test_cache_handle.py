"""What Python hands to the library: numbers as they are, and the pools where they lie now."""
import pytest
import torch

import tiled_attention_05_gb300 as fa
from test_cache import Setup, query


@pytest.mark.gpu
@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32 + 5, 2 ** 40])
def test_a_window_past_32_bits_hides_nothing(window):
    s = Setup([200, 30], 2, 64, 64, False, 16)
    Q = query(s, 4, 1)
    want = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths)
    got = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, window=window)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(fa.FAError):
        fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, window=5 - 2 ** 32)
