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
template <int KC, int ROWS>
void follow(int call, std::mt19937& rng) {
  constexpr bool PRE = ROWS == kPrefixRows;
  constexpr int kWarps = PRE ? 1 : 4, kMin = PRE ? kPrefixMinChunks : kCacheMinChunks;
  auto in = [&](int a, int b) { return a + (int)(rng() % (unsigned)(b - a + 1)); };
  CacheParams p = {};
  p.B = in(1, call % 3 ? 6 : 300);
  p.Hkv = in(1, 4);
  p.G = in(1, 9);
  p.T = in(1, call % 5 ? 4 : 40);
  p.page_log2 = in(4, 8);
  p.cols = in(0, call % 4 ? 12 : 200);
  p.S = in(PRE, 3);
  if (!PRE && p.S && prefix_apart(p.S, (long long)p.G * p.T * p.B)) p.S = 0;
  p.p_cols = in(0, 30);
  p.window = in(0, 2) ? 0 : in(1, 400);
  const int sms = in(1, 8);
  std::vector<int> lengths(p.B), plens(p.S + 1), starts(p.S + 1);
  for (int& n : lengths) n = in(-3, (p.cols << p.page_log2) + 5);
  for (int& n : plens) n = in(-3, (p.p_cols << p.page_log2) + 5);
  for (int s = 0; s <= p.S; ++s) starts[s] = in(s ? starts[s - 1] : 0, p.B);
  p.lengths = lengths.data();
  p.p_lengths = plens.data();
  p.p_starts = starts.data();
  const int rows = p.G * p.T, entries = PRE ? p.S : p.S + p.B;
  p.entries = entries;
  const CacheShape all = cache_shape(p.B, p.Hkv, rows, 64, KC == 32, (long long)p.cols << p.page_log2, p.S,
                                       (long long)p.p_cols << p.page_log2, sms);
  if (PRE && !all.apart) return;
  const CacheList shape = PRE ? all.pre : all.list;
  // the lists' areas follow one another
  auto fits = [&](const CacheList& l, long long n, int item_rows, size_t end) {
    return l.head + (n + 1) * sizeof(CacheHead) <= l.ml && l.ml + l.slots * item_rows * 8 <= l.part &&
           l.part + l.slots * item_rows * 64 * 4 <= end;
  };
  CHECK(fits(all.list, all.apart ? p.B : p.S + p.B, kCacheRows, all.apart ? all.pre.head : all.total));
  if (all.apart) CHECK(fits(all.pre, p.S, kPrefixRows, all.total));
  // the entries' places, as CTA 0 writes them
  std::vector<CacheHead> head(entries);
  long long total = 0;
  int items = 0;
  for (int e = 0; e < entries; ++e) {
    const CacheEntry n = cache_entry<KC>(p, e, true);
    head[e] = {total, items, n.chunks};
    total += (long long)p.Hkv * n.tiles(ROWS) * n.chunks;
    items += p.Hkv * n.tiles(ROWS);
  }
  CHECK(items <= shape.items);
  long long per = (total + shape.grid - 1) / shape.grid;
  if (per < kMin) per = kMin;
  CHECK(per * shape.grid >= total);
  std::set<std::tuple<int, int, int, int>> seen;
  std::map<long long, std::pair<int, int>> slots;  // slot -> item, CTA
  for (int cta = 0; cta < shape.grid; ++cta) {
    const long long begin = cta * per, end = begin + per < total ? begin + per : total;
    if (begin >= end) break;
    CacheCursor<KC, ROWS> it;
    it.e = 0;
    while (!(head[it.e].chunks && begin < head[it.e].work + (long long)p.Hkv * cache_entry<KC>(p, it.e, true).tiles(ROWS) * head[it.e].chunks))
      ++it.e;
    it.n = cache_entry<KC>(p, it.e, true);
    const long long into = begin - head[it.e].work;
    const int o = (int)(into / it.n.chunks);
    it.at = begin;
    it.c = (int)(into % it.n.chunks);
    it.h = o / it.n.tiles(ROWS);
    it.r = o % it.n.tiles(ROWS);
    int item = head[it.e].item + o;
    CacheCursor<KC, ROWS> warp[4] = {it, it, it, it};
    for (int w = 1; w < kWarps; ++w) warp[w].advance(p, true, w);
    while (it.at < end) {
      const long long left = end - it.at;
      const int c_end = left < it.n.chunks - it.c ? it.c + (int)left : it.n.chunks;
      CHECK(item == head[it.e].item + it.h * it.n.tiles(ROWS) + it.r);
      CHECK(item + cta < shape.slots);
      CHECK(slots.emplace((long long)item + cta, std::make_pair(item, cta)).second);
      for (int c = it.c; c < c_end; ++c) {
        CHECK(seen.insert({it.e, it.h, it.r, c}).second);
        // the warp whose turn it is stands there
        CacheCursor<KC, ROWS>& w = warp[(it.at + (c - it.c) - begin) % kWarps];
        CHECK(w.e == it.e && w.h == it.h && w.r == it.r && w.c == c && w.at == it.at + (c - it.c));
        const int key = (w.n.chunk0 + c) * KC;
        CHECK(key >= 0 && key < w.n.keys && (key >> p.page_log2) < (w.e < p.S ? p.p_cols : p.cols));
        w.advance(p, true, kWarps);
      }
      item += c_end == it.n.chunks;
      const int old = it.e;
      it.advance(p, true, c_end - it.c);
      for (int e = old + 1; e < it.e && e < entries; ++e) item += p.Hkv * cache_entry<KC>(p, e, true).tiles(ROWS);
    }
  }
  CHECK((long long)seen.size() == total);
  for (int e = 0; e < entries; ++e) {
    const CacheEntry n = cache_entry<KC>(p, e, true);
    for (int h = 0; h < p.Hkv; ++h)
      for (int row = 0; row < n.rows; ++row) {
        const CacheSlots l = cache_slots(head[e], n.rows, ROWS, h, row, per);
        CHECK((l.n > 0) == (n.chunks > 0) && l.row == row % ROWS);
        for (int i = 0; i < l.n; ++i) {
          CHECK(slots.count(l.slot + i));
          CHECK(slots[l.slot + i].first == head[e].item + h * n.tiles(ROWS) + row / ROWS);
          if (i) CHECK(slots[l.slot + i].second == slots[l.slot + i - 1].second + 1);
        }
        if (l.n) {  // no part before the first or after the last
          const int item = slots[l.slot].first;
          CHECK(!slots.count(l.slot - 1) || slots[l.slot - 1].first != item);
          CHECK(!slots.count(l.slot + l.n) || slots[l.slot + l.n].first != item);
        }
      }
  }
}

int main() {
  std::mt19937 rng(7);
  for (int call = 0; call < 400; ++call) {
    follow<32, kCacheRows>(call, rng);
    follow<16, kCacheRows>(call, rng);
    follow<kPrefixKeys, kPrefixRows>(call, rng);
  }
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
