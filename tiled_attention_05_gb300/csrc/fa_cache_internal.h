// Shared by the cache's translation units: the problem as the kernels see it,
// the walk over its work and the workspace of the attention.
#pragma once
#include <cstdint>

#include "fa_internal.h"
#ifdef __CUDACC__
#include "sm103_ptx.cuh"
#define FA_WALK __device__ __forceinline__
#else  // (the walk over the work also compiles for the host, where a test follows it)
#define FA_WALK inline
#endif

namespace fa {

constexpr int kCacheRows = 16;      // query rows of an item: one MMA's
constexpr int kCacheWarps = 4;      // warps of a CTA; each walks every fourth chunk of its keys
constexpr int kCacheCtasPerSm = 2;
// A CTA gets this many chunks of keys at least: two a warp, which is what setting it up
// and joining its part is worth.
constexpr int kCacheMinChunks = 8;

// One entry of the work list: the prefix of a group of sequences (entries 0 .. S - 1) or
// the own keys of sequence e - S.  An item is one (entry, kv head, tile of 16 rows).
struct CacheHead {
  long long work;  // chunks of all entries before this one
  int item;        // items of all entries before this one
  int chunks;      // of one item of this entry
};

struct CacheParams {
  const uint8_t *K, *V;
  const float *k_scale, *v_scale;
  const uint16_t* Q;
  const int *tables, *lengths;
  const int *p_tables, *p_lengths, *p_starts;  // S groups (p_starts NULL: one of all sequences)
  const float* slopes;
  uint16_t* O;
  float* L;
  CacheHead* head;  // [S + B + 1]; the last one's work: chunks a CTA
  float *ml, *part; // [slots][16][2], [slots][16][dv]
  int* status;
  int B, Hq, Hkv, G, T, pages, page_log2, cols, S, p_cols, window;
  int capped, min_chunks;
  float scale_log2;
  CapParams cap;
};

// The attention kernels, by the type of the cache, and the join of their parts.
cudaError_t launch_cache_attn_e4m3(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream);
cudaError_t launch_cache_attn_bf16(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream);
cudaError_t launch_cache_join(const CacheParams& p, int dv, cudaStream_t stream);

// Keys of a chunk, the unit of the walk: what one warp holds in one stage of its ring
// (8 KB at heads of 128).
constexpr int cache_chunk_keys(bool quantised) { return quantised ? 32 : 16; }

// Slots of the workspace and CTAs of a call, from what the host knows.  A part's slot is
// its item's ordinal + its CTA's: walking through the list, each next part raises one of
// the two, so that no two parts share one.
struct CacheShape {
  long long items;  // at most (a prefix has the rows of its sequences: 16 to an item, one
                    // item a group more for the remainders)
  int grid;
  size_t ml, part, total;  // byte offsets (the heads are at 0), size
};
inline CacheShape cache_shape(long long B, long long Hkv, long long rows, int dv, bool quantised, long long capacity,
                              long long groups, long long prefix_capacity, int sms) {
  CacheShape s;
  const long long kc = cache_chunk_keys(quantised), tiles = (rows + kCacheRows - 1) / kCacheRows;
  const long long p_tiles = groups ? groups + rows * B / kCacheRows : 0;
  s.items = Hkv * (B * tiles + p_tiles);
  const long long chunks = Hkv * (B * tiles * ((capacity + kc - 1) / kc) + p_tiles * ((prefix_capacity + kc - 1) / kc));
  const long long want = (chunks + kCacheMinChunks - 1) / kCacheMinChunks, most = (long long)kCacheCtasPerSm * sms;
  s.grid = (int)(want < 1 ? 1 : want < most ? want : most);
  const size_t slots = (size_t)(s.items + s.grid);
  s.ml = ((size_t)(groups + B + 1) * sizeof(CacheHead) + 255) / 256 * 256;
  s.part = s.ml + (slots * kCacheRows * 2 * sizeof(float) + 255) / 256 * 256;
  s.total = s.part + slots * kCacheRows * dv * sizeof(float);
  return s;
}

FA_WALK int cache_ld(const int* a) {
#ifdef __CUDACC__
  return __ldg(a);
#else
  return *a;
#endif
}
FA_WALK int cache_clamp(int x, int top) { return x < 0 ? 0 : x < top ? x : top; }

struct CacheEntry {
  int first;   // first sequence of the group, or the sequence
  int rows;    // query rows of one kv head
  int keys;    // keys of the entry
  int chunk0;  // first chunk that any row may see
  int chunks;  // from there on
  FA_WALK int tiles() const { return (rows + kCacheRows - 1) / kCacheRows; }
};

FA_WALK int cache_length(const CacheParams& p, int b) {
  return cache_clamp(cache_ld(p.lengths + b), p.cols << p.page_log2);
}
FA_WALK int cache_group_start(const CacheParams& p, int s) {
  return p.p_starts ? cache_ld(p.p_starts + s) : s ? p.B : 0;
}

template <int KC>
FA_WALK CacheEntry cache_entry(const CacheParams& p, int e, bool groups_ok) {
  CacheEntry n;
  int first_key;  // the first that a row may see, with a window
  if (e < p.S) {
    n.first = cache_group_start(p, e);
    n.rows = groups_ok ? (cache_group_start(p, e + 1) - n.first) * p.G * p.T : 0;
    n.keys = cache_clamp(cache_ld(p.p_lengths + e), p.p_cols << p.page_log2);
    first_key = n.keys - p.window + 1;  // (the first row of all stands behind the prefix)
  } else {
    n.first = e - p.S;
    n.rows = p.G * p.T;
    n.keys = cache_length(p, n.first);
    first_key = (n.keys > p.T ? n.keys - p.T : 0) - p.window + 1;
  }
  n.chunk0 = p.window && first_key > 0 ? first_key / KC : 0;
  n.chunks = n.rows > 0 ? (n.keys + KC - 1) / KC - n.chunk0 : 0;
  if (n.chunks < 0) n.chunks = 0;
  return n;
}

// A place in the list of chunks: that of chunk c of the item of tile r, kv head h, entry e.
struct CacheCursor {
  long long at;  // in the whole list
  int e, h, r, c;
  CacheEntry n;
  template <int KC>
  FA_WALK void advance(const CacheParams& p, bool groups_ok, int k) {
    at += k;
    c += k;
    while (c >= n.chunks) {
      c -= n.chunks;
      if (++r < n.tiles()) continue;
      r = 0;
      if (++h < p.Hkv) continue;
      h = 0;
      do {
        if (++e >= p.S + p.B) {  // the list's end: stay there
          n.chunks = 0x7fffffff;
          return;
        }
        n = cache_entry<KC>(p, e, groups_ok);
      } while (n.chunks == 0);
    }
  }
};

// Where the join finds the parts of row `row` of an entry's kv head h: `n` slots from
// `slot` on (`per`: chunks a CTA).
struct CacheParts {
  long long slot;
  int n, row;  // parts, row within the tile
};
FA_WALK CacheParts cache_parts(const CacheHead& e, int rows, int h, int row, long long per) {
  CacheParts l = {0, 0, row % kCacheRows};
  if (e.chunks == 0) return l;
  const int o = h * ((rows + kCacheRows - 1) / kCacheRows) + row / kCacheRows;
  const long long at = e.work + (long long)o * e.chunks, c0 = at / per, c1 = (at + e.chunks - 1) / per;
  l.slot = (long long)e.item + o + c0;
  l.n = (int)(c1 - c0) + 1;
  return l;
}

#ifdef __CUDACC__
// Whether the groups' starts are a list of disjoint runs of sequences.  Every thread of
// the CTA gets the answer.
__device__ __forceinline__ bool cache_groups_ok(const CacheParams& p) {
  bool ok = true;
  if (p.p_starts)
    for (int s = threadIdx.x; s < p.S; s += blockDim.x) {
      const int a = __ldg(p.p_starts + s), z = __ldg(p.p_starts + s + 1);
      ok = ok && a >= 0 && a <= z && z <= p.B;
    }
  return p.S == 0 || __syncthreads_and(ok);
}

// An index that does not fit: the device status word says so (a timeout stays).
__device__ __forceinline__ void cache_bad(int* status) { atomicCAS(status, 0, fa_ptx::DEV_BAD_TABLE); }
#endif

}  // namespace fa
