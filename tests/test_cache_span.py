"""The keys that fa_cache_attention walks are those that some row sees: with a window the
first one hangs on where the rows of a sequence, or of all sequences that share a prefix,
stand.  On the host the library's own header is compiled with g++ and compared with the
definition; on the GPU what lies before the window has no pages any more."""
import os
import shutil
import subprocess

import pytest

import tiled_attention_05_gb300 as fa
from test_cache import Setup, check, query

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tiled_attention_05_gb300", "csrc")
CUDA_INC = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "fa_cache_internal.h"
using namespace fa;

#define CHECK(x) do { if (!(x)) { std::printf("failed: %s (call %d)\n", #x, call); std::exit(1); } } while (0)

int hidden_prefixes = 0, partly = 0;
template <int KC>
void follow(int call, std::mt19937& rng) {
  auto in = [&](int a, int b) { return a + (int)(rng() % (unsigned)(b - a + 1)); };
  CacheParams p = {};
  p.B = in(1, 12);
  p.Hkv = 1;
  p.G = in(1, 3);
  p.T = in(1, 6);
  p.page_log2 = in(4, 8);
  p.cols = in(0, 20);
  p.S = in(1, 4);
  p.p_cols = in(0, 20);
  p.window = in(0, 3) ? in(1, call % 2 ? 40 : 2000) : 0;
  std::vector<int> lengths(p.B), plens(p.S), starts(p.S + 1);
  const int most = in(0, (p.cols << p.page_log2) + 5);
  for (int& n : lengths) n = in(0, 3) ? in(-2, most) : in(-1, p.T);
  for (int& n : plens) n = in(-3, (p.p_cols << p.page_log2) + 5);
  for (int s = 0; s <= p.S; ++s) starts[s] = in(s ? starts[s - 1] : 0, p.B);
  p.lengths = lengths.data();
  p.p_lengths = plens.data();
  p.p_starts = starts.data();
  p.entries = p.S + p.B;
  for (int e = 0; e < p.entries; ++e) {
    const CacheEntry n = cache_entry<KC>(p, e);
    const bool prefix = e < p.S;
    const int first = prefix ? starts[e] : e - p.S, end = prefix ? starts[e + 1] : e - p.S + 1;
    int from = 1 << 30;  // the first key that any row sees
    for (int b = first; b < end; ++b) {
      const int own = cache_clamp(lengths[b], p.cols << p.page_log2);
      for (int t = 0; t < p.T; ++t) {
        const int pos = own - p.T + t, at = prefix ? n.keys + pos : pos;
        if (pos < 0) continue;
        for (int j = 0; j < n.keys && j <= at; ++j)
          if (!p.window || at - j < p.window) {
            from = j < from ? j : from;
            break;
          }
      }
    }
    CHECK(n.keys == cache_clamp(prefix ? plens[e] : lengths[e - p.S], (prefix ? p.p_cols : p.cols) << p.page_log2));
    if (from >= n.keys) {  // (without a window an empty sequence's prefix is walked)
      CHECK(n.chunks == 0 || (prefix && !p.window) || n.keys == 0);
      hidden_prefixes += prefix && p.window && n.keys > 0 && n.rows > 0;
    } else {
      CHECK(n.chunk0 == from / KC && n.chunk0 + n.chunks == (n.keys + KC - 1) / KC);
      partly += prefix && from > 0;
    }
  }
}

int main() {
  std::mt19937 rng(11);
  for (int call = 0; call < 3000; ++call) {
    follow<kCacheKeys>(call, rng);
    follow<kPrefixKeys>(call, rng);
  }
  const int call = -1;
  CHECK(hidden_prefixes > 300 && partly > 300);
  // the largest numbers stay in 32 bits
  CacheParams p = {};
  int length = 1 << 30;
  p.B = p.S = p.Hkv = p.G = p.T = p.entries = 1;
  p.page_log2 = 8, p.cols = p.p_cols = 1 << 22;
  p.lengths = p.p_lengths = &length;
  const int windows[][2] = {{1, 0}, {1 << 30, 0}, {(1 << 30) + 1, 1}, {(1 << 30) + 17, 2}, {0x7fffffff, 1 << 26}};
  for (auto& w : windows) {  // window, chunks: the row stands at 2^31 - 1, keys end at 2^30
    p.window = w[0];
    CHECK(cache_prefix<kCacheKeys>(p, 0).chunks == w[1]);
  }
  std::printf("ok\n");
}
"""


def test_the_span_is_what_some_row_sees(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA_INC, "cuda.h")):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "span.cpp", tmp_path / "span"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", f"-I{CUDA_INC}", str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout.strip() == "ok"


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("lens, starts, T, window", [
    ([50, 61], None, 1, 120),                        # the window begins inside the prefix
    ([50, 61, 77] * 10, None, 1, 120),
    ([50, 61], None, 3, 120),
    ([150, 161, 300] * 10, None, 1, 120),            # ... and behind it
    ([150, 161, 300], None, 5, 120),
    ([0, 150, 0, 131], None, 2, 100),                # (an empty sequence has no rows that see anything)
    ([0, 90, 200, 61] * 8, None, 2, 100),
    ([70, 300, 70, 90, 0, 0] * 8, [0, 1, 2, 4, 6, 20, 33, 48], 1, 100),
    ([30 + 3 * k for k in range(80)], list(range(0, 81, 2)), 1, 100),  # many groups
])
def test_pages_behind_all_rows_may_be_dropped(lens, starts, T, window, quant):
    """Windowed pages of a prefix that the rows have all left are no longer the cache's: -1."""
    groups = len(starts) - 1 if starts else 1
    s = Setup(lens, 2, 64, 64, quant, 16, [400] * groups, starts)
    Q = query(s, 8, T)
    dropped, ends = s.p_tables.clone(), starts or [0, len(lens)]
    for g in range(groups):
        at = [max(n - T, 0) for n in lens[ends[g]:ends[g + 1]] if n > 0]
        dropped[g, :max(400 + min(at) - window + 1, 0) // 16 if at else 400] = -1
    prefix = (dropped, *s.prefix[1:])
    O, L = fa.fa_cache_attention(Q, s.cache, s.tables, s.lengths, prefix=prefix, window=window)
    assert fa.fa_last_device_status() == fa.FA_OK
    check(s, Q, O, L, window=window)
