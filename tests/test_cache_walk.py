"""The walk of fa_cache_attention over its list of work, followed on the host: the
library's own header compiled with g++.  Every chunk of keys of every item is visited
once, by one CTA; no two parts of the workspace share a slot and none lies outside of
it; and the join finds exactly the parts that were written."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tiled_attention_05_gb300", "csrc")
CUDA_INC = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <vector>
#include "fa_cache_internal.h"
using namespace fa;

#define CHECK(x) do { if (!(x)) { std::printf("failed: %s (call %d)\n", #x, call); std::exit(1); } } while (0)

// ROWS 16: own keys and prefixes in one list; 256: the prefixes' own list
int wholes = 0, bundles = 0, calls[2];
template <int KC, int ROWS, bool FEW>
void follow(int call, std::mt19937& rng) {
  constexpr bool PRE = ROWS == kPrefixRows;
  constexpr int kWarps = PRE ? 1 : 4, kItem = PRE ? kPrefixItem : cache_item(FEW), kMin = PRE ? kPrefixMinChunks : kCacheMinChunks;
  auto in = [&](int a, int b) { return a + (int)(rng() % (unsigned)(b - a + 1)); };
  CacheParams p = {};
  p.B = in(1, call % 3 ? 6 : 300);
  p.Hkv = in(1, 4);
  p.G = in(1, 9);
  p.T = in(1, call % 5 ? 4 : 40);
  p.page_log2 = in(4, 8);
  p.cols = in(0, call % 4 ? 12 : 200);
  p.S = in(PRE, 3);
  if (!PRE && p.S && prefix_apart(p.S, (long long)p.G * p.T * p.B, call % 2, 64)) p.S = 0;
  p.p_cols = in(0, 30);
  p.window = in(0, 2) ? 0 : in(1, 400);
  const int sms = in(1, call % 2 ? 8 : 60);
  std::vector<int> lengths(p.B), plens(p.S + 1), starts(p.S + 1);
  for (int& n : lengths) n = in(-3, (p.cols << p.page_log2) + 5);
  for (int& n : plens) n = in(-3, (p.p_cols << p.page_log2) + 5);
  for (int s = 0; s <= p.S; ++s) starts[s] = in(s ? starts[s - 1] : 0, p.B);
  p.lengths = lengths.data();
  p.p_lengths = plens.data();
  p.p_starts = starts.data();
  const int rows = p.G * p.T, entries = PRE ? p.S : p.S + p.B;
  p.entries = entries;
  const CacheShape all = cache_shape(p.B, p.Hkv, rows, 64, call % 2, (long long)p.cols << p.page_log2, p.S,
                                       (long long)p.p_cols << p.page_log2, sms);
  if (PRE && !all.apart) return;
  if (!PRE && cache_few(rows, p.S > 0) != FEW) return;
  ++calls[FEW];
  p.whole = all.whole;
  wholes += all.whole;
  const CacheList shape = PRE ? all.pre : all.list;
  // the lists' areas follow one another
  auto fits = [&](const CacheList& l, long long n, int item_rows, size_t end) {
    return l.head + (n + 1) * sizeof(CacheHead) <= l.ml && l.ml + l.slots * item_rows * 8 <= l.part &&
           l.part + l.slots * item_rows * 64 * 4 <= end;
  };
  if (all.whole) CHECK(all.total == 0 && p.S == 0);
  else CHECK(fits(all.list, all.apart ? p.B : p.S + p.B, kCacheRows, all.apart ? all.pre.head : all.total));
  if (all.apart) CHECK(fits(all.pre, p.S, kPrefixRows, all.total));
  // the entries' places, as CTA 0 writes them (in bundles of tiles)
  const int bundle = PRE ? cache_bundle(p.S, cache_prefix<kPrefixKeys>(p, 0).tiles(kPrefixRows), shape.grid) : 1;
  bundles += bundle > 1;
  std::vector<CacheHead> head(entries);
  long long total = 0, chunks = 0;
  int items = 0;
  for (int e = 0; e < entries; ++e) {
    const CacheEntry n = cache_entry<KC>(p, e);
    head[e] = {(int)total, items, n.chunks};
    if (n.chunks || p.whole) total += (long long)p.Hkv * (n.tiles(ROWS) / bundle) * (n.chunks + kItem);
    chunks += (long long)p.Hkv * (n.tiles(ROWS) / bundle) * n.chunks;
    items += p.Hkv * (n.tiles(ROWS) / bundle);
  }
  CHECK(all.fits && items <= shape.items);
  const int ctas = shape.grid / bundle;
  long long per = (total + ctas - 1) / ctas;
  if (per < kMin) per = kMin;
  CHECK(per * ctas >= total);
  std::set<std::tuple<int, int, int, int>> seen;
  std::map<long long, std::pair<int, int>> slots;  // slot -> item, CTA
  std::set<int> items_seen;
  for (int cta = 0; cta < ctas; ++cta) {
    const long long begin = cta * per, end = begin + per < total ? begin + per : total;
    if (begin >= end) break;
    using Cursor = CacheCursor<KC, ROWS, kItem>;
    int e = 0;
    while (!((head[e].chunks || p.whole) && begin < head[e].work + (long long)p.Hkv * (cache_entry<KC>(p, e).tiles(ROWS) / bundle) * (head[e].chunks + kItem))) ++e;
    Cursor it;
    it.start(p, bundle, e, head[e].item, (int)begin, (int)(begin - head[e].work));
    for (; it.at < end; it.next(p)) {
      const int c_end = it.end(p, (int)end);
      CHECK(p.whole ? it.c == 0 && c_end == it.n.chunks : it.c < c_end);
      if (p.whole) CHECK(items_seen.insert(it.item).second);
      CHECK(it.item == head[it.e].item + it.h * it.tiles() + it.r);
      CHECK(it.at == head[it.e].work + (it.h * it.tiles() + it.r) * (it.n.chunks + kItem) + it.c);
      for (int tile = 0; tile < bundle; ++tile) {
        const long long slot = ((long long)it.item + cta) * bundle + tile;
        CHECK(slot < shape.slots);
        CHECK(slots.emplace(slot, std::make_pair(it.item * bundle + tile, cta)).second);
      }
      for (int c = it.c; c < c_end; ++c) {
        CHECK(seen.insert({it.e, it.h, it.r, c}).second);
        const int key = (it.n.chunk0 + c) * KC;
        CHECK(key >= 0 && key < it.n.keys && (key >> p.page_log2) < (it.e < p.S ? p.p_cols : p.cols));
      }
    }
    // each warp's chunks, as the loads walk ahead: the same that it meets item by item
    if (!PRE)
      for (int warp = 0; warp < kWarps; ++warp) {
        Cursor ld;
        ld.start(p, bundle, e, head[e].item, (int)begin, (int)(begin - head[e].work));
        if (ld.at >= end) break;
        Cursor use = ld;
        int lc = ld.c + warp, lc_end = ld.end(p, (int)end), turn = 0;
        auto next_load = [&](int step) {
          lc += step;
          while (lc >= lc_end) {
            ld.next(p);
            if (ld.at >= end) return;
            ++turn;
            lc = ld.c + ((warp - turn) & 3);
            lc_end = ld.end(p, (int)end);
          }
        };
        next_load(0);
        int t = 0;
        for (; use.at < end; use.next(p), ++t)
          for (int c = use.c + ((warp - t) & 3); c < use.end(p, (int)end); c += 4) {
            CHECK(lc < lc_end && ld.item == use.item && lc == c);
            next_load(4);
          }
        CHECK(lc >= lc_end);
      }
  }
  CHECK((long long)seen.size() == chunks);
  if (p.whole) {
    CHECK((int)items_seen.size() == items);
    return;
  }
  for (int e = 0; e < entries; ++e) {
    const CacheEntry n = cache_entry<KC>(p, e);
    for (int h = 0; h < p.Hkv; ++h)
      for (int row = 0; row < n.rows; ++row) {
        const CacheSlots l = cache_slots(head[e], n.rows, ROWS, kItem, bundle, h, row, (int)per);
        CHECK((l.n > 0) == (n.chunks > 0) && l.row == row % ROWS);
        for (int i = 0; i < l.n; ++i) {
          const long long at = l.slot + (long long)i * l.step;
          CHECK(slots.count(at));
          CHECK(slots[at].first == head[e].item * bundle + h * n.tiles(ROWS) + row / ROWS);
          if (i) CHECK(slots[at].second == slots[at - l.step].second + 1);
        }
        if (l.n) {  // no part before the first or after the last
          const int item = slots[l.slot].first;
          const long long after = l.slot + (long long)l.n * l.step, before = l.slot - l.step;
          CHECK(!slots.count(before) || slots[before].first != item);
          CHECK(!slots.count(after) || slots[after].first != item);
        }
      }
  }
}

int main() {
  std::mt19937 rng(7);
  for (int by : {1, 2, 3, 5, 7, 16, 255, 1000003, (1 << 30) - 1, 1 << 30})
    for (int k = 0; k < 2000; ++k) {
      const int call = by, n = k < 100 ? k : (int)(rng() & ((1u << 30) - 1)), d = Divide::of(by)(n);
      CHECK(d == n / by);
      const int m = n / by * by;  // at a multiple, and before one
      CHECK(Divide::of(by)(m) == m / by && (m == 0 || Divide::of(by)(m - 1) == (m - 1) / by));
    }
  for (int call = 0; call < 600; ++call) {
    follow<kCacheKeys, kCacheRows, true>(call, rng);
    follow<kCacheKeys, kCacheRows, false>(call, rng);
    follow<kPrefixKeys, kPrefixRows, false>(call, rng);
  }
  const int call = -1;
  // shares of lists of any size, for fewer CTAs than the grid has, too
  for (int k = 0; k < 3000; ++k) {
    const int all = k < 50 ? k : (int)(rng() % (1u << (10 + k % 21))), grid = 1 + (int)(rng() % 600), least = 1 + k % 8;
    const unsigned ctas = 1 + rng() % (unsigned)(k % 3 ? grid : k % 5 + 1);
    long long at = 0, size = 0;
    for (int cta = 0; cta < (grid > (int)ctas ? grid : (int)ctas); ++cta) {
      int begin, end;
      const int per = cache_cut(all, ctas, least, cta, &begin, &end);
      CHECK(begin == at && begin <= end && end <= all && end - begin <= per && per >= least);
      CHECK(end == all || end - begin == per);
      CHECK(cta == 0 || per == size);
      at = end;
      size = per;
    }
    CHECK(at == all);
  }
  CHECK(wholes > 10 && bundles > 10 && calls[0] > 100 && calls[1] > 100);
  std::printf("ok\n");
}
"""


def test_every_chunk_once_and_every_part_found(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA_INC, "cuda.h")):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", f"-I{CUDA_INC}", str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout.strip() == "ok"
