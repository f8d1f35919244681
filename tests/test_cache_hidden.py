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


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("lens", [[1, 2, 3, 17] * 8, [1, 3]])
@pytest.mark.parametrize("page, window", [(16, 100), (32, 1), (16, 205), (256, 300)])
def test_pages_before_the_window_may_be_dropped(lens, quant, page, window):
    """Pages of a prefix that the window hides from every row are no longer the cache's: their
    places in the table hold -1, and what lay in shared memory before is not taken for them."""
    s = Setup(lens, 2, 64, 64, quant, page, [700])
    Q = query(s, 8, 1)
    other = Setup(lens, 2, 64, 64, quant, page, [700])
    for x in (other.cache.K, other.cache.V):
        x.view(torch.uint8).fill_(0x7f)  # NaN in both types
    dropped = s.p_tables.clone()
    dropped[:, :(700 - window + 1) // page] = -1  # (a row at its first position sees the furthest)
    prefix = (dropped, *s.prefix[1:])
    for mods in (dict(), dict(softcap=20.0, slopes=slopes_of(8))):
        fa.fa_cache_attention(Q, other.cache, other.tables, other.lengths, prefix=other.prefix)
        O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=prefix, window=window, **mods)
        assert fa.fa_last_device_status() == fa.FA_OK
        check(s, Q, O, L, window=window, **mods)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_a_bad_page_of_a_prefix_is_its_groups_alone(page, quant):
    s = Setup([30] * 40, 1, 64, 64, quant, page, [700, 690], [0, 20, 40])
    Q = query(s, 4, 1)
    want = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix)
    for bad in (-1, 10 ** 6):
        tables = s.p_tables.clone()
        tables[0, 1] = bad
        for mods in (dict(), dict(window=720)):
            O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=(tables, *s.prefix[1:]), **mods)
            assert fa.fa_last_device_status() == fa.FA_ERR_BAD_TABLE
            if not mods:
                assert torch.equal(O[20:], want[0][20:]) and torch.equal(L[20:], want[1][20:])
    again = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    assert fa.fa_last_device_status() == fa.FA_OK


def spoil(x, table, page, keys, value):
    """``value`` in the rows of positions ``keys`` of one table."""
    p = torch.as_tensor(keys, device="cuda")
    x.view(torch.int16)[table.long()[p // page], :, p % page] = torch.tensor(value).to(bf).view(torch.int16).item()


@pytest.mark.gpu
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("dv", [64, 128])
def test_values_before_the_window(dv, T, value):
    """bf16: what a window hides from all rows may be anything, wherever the window begins in a
    chunk or a tile of keys."""
    s = Setup([90, 41, 300], 2, 64, dv, False, 16)
    Q = query(s, 8, T)
    clean = s.cache.V.clone()
    for window in (20, 21, 27, 36):
        want = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, window=window)
        check(s, Q, *want, window=window)
        for table, n in zip(s.tables, s.lens):
            spoil(s.cache.V, table, 16, list(range(n - T - window + 1)), value)
        got = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        s.cache.V.copy_(clean)


@pytest.mark.gpu
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("lens", [MANY, FEW])
@pytest.mark.parametrize("dv", [64, 128])
def test_values_of_a_prefix_before_the_window(dv, lens, value):
    s = Setup(lens, 2, 64, dv, False, 16, [700])
    Q = query(s, 8, 2)
    clean = s.cache.V.clone()
    for window, softcap in ((60, 0.0), (133, 0.0), (501, 0.0), (95, 20.0)):
        mods = dict(window=window, softcap=softcap)
        want = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, **mods)
        check(s, Q, *want, **mods)
        spoil(s.cache.V, s.p_tables[0], 16, list(range(700 + 28 - window + 1)), value)
        got = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, **mods)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        s.cache.V.copy_(clean)


@pytest.mark.gpu
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d, dv", [(64, 64), (128, 128), (64, 128)])
@pytest.mark.parametrize("Hq, T", [(2, 3), (8, 4), (6, 17)])
def test_values_that_some_rows_see(Hq, T, d, dv, value):
    """bf16: a value of the newest tokens, or one at the window's edge, reaches those rows that see
    it, in its channel; the others' results are as if it was not there."""
    s = Setup([90, 41, 300, 7], 2, d, dv, False, 16)
    Q = query(s, Hq, T)
    clean = s.cache.V.clone()
    for window, back in ((0, 1), (0, 2), (20, 1), (20, 20 + T // 2), (33, 34)):  # the key is the back-th from the end
        want = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, window=window)
        for b, n in enumerate(s.lens):
            if n >= back:
                spoil(s.cache.V[..., 5:6], s.tables[b], 16, [n - back], value)
                spoil(s.cache.V[..., dv - 3:dv - 2], s.tables[b], 16, [n - back], math.nan)
        got = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, window=window)
        assert torch.equal(got[1], want[1])
        for b, n in enumerate(s.lens):
            for t in range(T):
                far = n - T + t - (n - back)
                sees = n >= back and n - T + t >= 0 and far >= 0 and (not window or far < window)
                hit = torch.zeros(dv, dtype=torch.bool, device="cuda")
                hit[[5, dv - 3]] = sees
                assert torch.equal(got[0][b, :, t, ~hit], want[0][b, :, t, ~hit]), (window, back, b, t)
                assert not torch.isfinite(got[0][b, :, t, hit]).any()
        s.cache.V.copy_(clean)


@pytest.mark.gpu
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("dv", [64, 128])
def test_values_of_a_prefix_that_some_sequences_see(dv, value):
    """bf16, a prefix of few rows: the window hides its key 650 from some sequences."""
    lens, window = [30, 41, 42, 70, 2], 92
    s = Setup(lens, 2, 128, dv, False, 16, [700])
    Q = query(s, 4, 1)
    want = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, window=window)
    check(s, Q, *want, window=window)
    spoil(s.cache.V[..., 7:8], s.p_tables[0], 16, [650], value)
    got = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, window=window)
    hit = torch.zeros(dv, dtype=torch.bool, device="cuda")
    hit[7] = True
    assert torch.equal(got[1], want[1]) and torch.equal(got[0][..., ~hit], want[0][..., ~hit])
    for b, n in enumerate(lens):
        sees = 700 + n - 1 - 650 < window
        assert (~torch.isfinite(got[0][b, :, 0, 7]) if sees else got[0][b, :, 0, 7] == want[0][b, :, 0, 7]).all(), b


@pytest.mark.gpu
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("lens, starts, Hq, Hkv, T, d, dv, page", [
    ([30, 41, 42, 70, 2, 300] * 8, None, 8, 2, 1, 128, 128, 16),    # several tiles of rows
    ([30, 41, 42, 70, 2, 300], None, 8, 1, 1, 64, 128, 256),        # one: two parts of even and odd key tiles
    ([38, 45], None, 32, 2, 9, 128, 64, 64),                        # rows of one sequence differ, too
    ([30, 45, 300] * 60, list(range(0, 181, 3)), 64, 8, 1, 64, 64, 32),  # several items a CTA
    ([30, 45, 300] * 60, list(range(0, 181, 3)), 128, 8, 1, 128, 128, 32),
])
def test_values_of_a_prefix_that_some_rows_see(lens, starts, Hq, Hkv, T, d, dv, page, softcap, value):
    """bf16, prefixes of many rows: keys at the edges of the rows' windows, in several tiles."""
    window, groups = 292, len(starts) - 1 if starts else 1
    s = Setup(lens, Hkv, d, dv, False, page, [700] * groups, starts)
    Q = query(s, Hq, T)
    mods = dict(window=window, softcap=softcap)
    want = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, **mods)
    check(s, Q, *want, **mods)
    keys = {5: 409, 8: 450, dv - 1: 450, 0: 511, 33: 512, 40: 699}  # channel: key
    hurt = [g for g in range(groups) if groups == 1 or g % 7 == 3]
    for g in hurt:
        for c, key in keys.items():
            spoil(s.cache.V[..., c:c + 1], s.p_tables[g], page, [key], value)
    got = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, **mods)
    assert torch.equal(got[1], want[1])
    hit = torch.zeros(len(lens), T, dv, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for t in range(T):
            for c, key in keys.items():
                hit[b, t, c] = s.group(b) in hurt and n - T + t >= 0 and 700 + n - T + t - key < window
    hit = hit[:, None].expand_as(got[0])
    assert hit.any() and torch.equal(got[0][~hit], want[0][~hit])
    assert not torch.isfinite(got[0][hit]).any()


@pytest.mark.gpu
def test_captured_windowed_prefix_is_replayed_with_other_values():
    """Two graphs with one workspace, bf16, many rows, a window: replayed with values that are finite
    and not, with other lengths, and the workspace's neighbours left alone."""
    s = Setup([30, 41, 42, 70, 2, 300] * 8, 2, 128, 128, False, 16, [700])
    Q, window = query(s, 8, 1), 292
    lengths = s.lengths.clone()
    need = fa.fa_cache_attention_workspace_bytes(Q, s.cache, s.tables, s.prefix)
    ws = torch.full((need + 4096,), 0xff, dtype=torch.uint8, device="cuda")

    def step():
        return fa.fa_cache_attention(Q, s.cache, s.tables, lengths, prefix=s.prefix, window=window, workspace=ws[:need])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    clean, lens = s.cache.V.clone(), list(s.lens)
    for k in range(6):
        graph, (O, L) = graphs[k % 2]
        s.lens = [max(n - 3 * k, 0) for n in lens]
        lengths.copy_(torch.tensor(s.lens, dtype=torch.int32))
        s.cache.V.copy_(clean)
        if k % 3 == 1:
            spoil(s.cache.V[..., 9:10], s.p_tables[0], 16, [450], math.nan)
        graph.replay()
        torch.cuda.synchronize()
        sees = torch.tensor([k % 3 == 1 and n > 0 and 700 + n - 1 - 450 < window for n in s.lens], device="cuda")
        assert (torch.isfinite(O[..., 9]) != sees[:, None, None]).all()
        O[..., 9] = O[..., 9].nan_to_num(0.0)
        s.cache.V.copy_(clean)
        if k % 3 != 1:
            check(s, Q, O, L, window=window)
        else:
            want = fa.fa_cache_attention(Q, s.cache, s.tables, lengths, prefix=s.prefix, window=window)
            keep = ~sees[:, None, None, None].expand_as(O) | (torch.arange(128, device="cuda") != 9)
            assert torch.equal(O[keep], want[0][keep]) and torch.equal(L, want[1])
    assert (ws[need:] == 0xff).all()
    assert fa.fa_last_device_status() == fa.FA_OK


@pytest.mark.gpu
def test_windowed_prefixes_on_two_streams():
    sets = [Setup([30 + k, 41, 70, 2, 300] * 8, 2, 64, 128, False, 16, [700], seed=k) for k in range(2)]
    Qs, window = [query(s, 8, 1) for s in sets], 292
    for s in sets:
        spoil(s.cache.V[..., 3:4], s.p_tables[0], 16, [450], math.nan)
    want = [fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, window=window) for s, Q in zip(sets, Qs)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=s.prefix, window=window, stream=t)
               for s, Q, t in zip(sets, Qs, streams)]
    torch.cuda.synchronize()
    for (O, L), (Ow, Lw), s in zip(got, want, sets):
        assert torch.equal(O.view(torch.int16), Ow.view(torch.int16)) and torch.equal(L, Lw)
        seen = torch.tensor([700 + n - 1 - 450 < window for n in s.lens], device="cuda")
        assert (torch.isfinite(O[:, :, 0, 3]) != seen[:, None]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("page, window, T", [(16, 1, 1), (16, 40, 3), (128, 130, 1), (32, 31, 5)])
def test_own_pages_before_the_window_may_be_dropped(page, window, T, quant):
    s = Setup([300, 41, 1, 129, 700], 2, 64, 64, quant, page)
    Q = query(s, 8, T)
    tables = s.tables.clone()
    for b, n in enumerate(s.lens):
        tables[b, :max(max(n - T, 0) - window + 1, 0) // page] = -1
    O, L = fa.fa_cache_attention(Q, s.cache, tables, s.lengths, window=window)
    assert fa.fa_last_device_status() == fa.FA_OK
    check(s, Q, O, L, window=window)
