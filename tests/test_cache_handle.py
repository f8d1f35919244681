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


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["K", "V", "k_scale", "v_scale"])
def test_a_pool_that_moved_is_refused(name):
    """The library is given addresses; a tensor that was given other memory since has another one."""
    s = Setup([50, 30], 2, 64, 64, True, 16)
    Q = query(s, 4, 1)
    x = torch.zeros(2, 2, 1, 64, device="cuda").to(torch.bfloat16)
    calls = [lambda: fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths),
             lambda: fa.fa_cache_read(s.cache, s.tables, s.lengths, 10),
             lambda: fa.fa_cache_write(s.cache, x, x, s.tables, s.lengths - 1)]
    for call in calls:
        call()
    pool = getattr(s.cache, name)
    kept = pool.data
    pool.data = pool.data.clone()
    for call in calls:
        with pytest.raises(ValueError, match="moved"):
            call()
    pool.data = kept
    for call in calls:
        call()


@pytest.mark.gpu
def test_a_pool_of_other_sizes_is_refused():
    s = Setup([50, 30], 2, 64, 64, False, 16)
    Q = query(s, 4, 1)
    fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths)
    s.cache.K.data = s.cache.K.data[:1]  # (the same address)
    with pytest.raises(ValueError, match="moved"):
        fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths)
