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

// The attention's work is one list of chunks of keys, cut into equal shares, one for
// each CTA.  An item of it is one (entry, kv head, tile of query rows); an entry is the
// prefix of a group of sequences (entries 0 .. S - 1), or the own keys of a sequence
// (entries S .. S + B - 1).
constexpr int kCacheRows = 16;      // query rows of an item: one MMA's
constexpr int kCacheWarps = 4;      // warps of a CTA; each walks every fourth chunk of its keys
constexpr int kCacheCtasPerSm = 2;
// A CTA gets this many chunks of keys at least: two a warp, which is what setting it up
// and joining its part is worth.
constexpr int kCacheMinChunks = 8;
// Prefixes of many rows have a list of their own (fa_cache_prefix_kernel), with items of
// two tiles of 128 rows and chunks of 128 keys.
constexpr int kPrefixRows = 256, kPrefixKeys = 128, kPrefixMinChunks = 4;

struct CacheHead {
  long long work;  // chunks of all entries before this one
  int item;        // items of all entries before this one
  int chunks;      // of one item of this entry
};
// Parts of items (of `rows` rows each) that a join adds up.
struct CacheParts {
  CacheHead* head;  // [entries + 1]; the last one's work: chunks a CTA
  float *ml, *part; // [slots][rows][2]: reference and sum; [slots][rows][dv]: unnormalised O
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
  CacheParts parts;
  int* status;
  int B, Hq, Hkv, G, T, pages, page_log2, cols, S, p_cols, window;
  int entries;     // of the list: S + B, or S (prefixes alone)
  int joined;      // whole items too leave their part for the join
  int capped, min_chunks;
  float scale_log2;
  CapParams cap;
};
// What the join adds to the own keys' parts: those of the prefixes.
struct CacheJoin {
  CacheParams p;       // p.S = 0: no prefixes; parts: of the own keys
  int own;             // entry of sequence 0 in its list
  int own_entries;     // of that list
  CacheParts pre;      // parts of the prefixes, in items of pre_rows rows
  int pre_rows, pre_entries;
};

// The kernels, by the type of the cache, and the join of their parts.
cudaError_t launch_cache_attn_e4m3(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream);
cudaError_t launch_cache_attn_bf16(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream);
cudaError_t launch_cache_prefix_e4m3(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream);
cudaError_t launch_cache_prefix_bf16(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream);
cudaError_t launch_cache_join(const CacheJoin& j, int dv, cudaStream_t stream);

// Keys of a chunk, the unit of the walk: what one warp holds in one stage of its ring
// (8 KB at heads of 128).
constexpr int cache_chunk_keys(bool quantised) { return quantised ? 32 : 16; }

// Whether the prefixes go through the kernel that takes 128 rows at a time (`rows`: those
// of all sequences' kv heads).
inline bool prefix_apart(long long groups, long long rows) { return groups > 0 && rows > 32 * groups; }

// Slots of the workspace and CTAs of a call, from what the host knows.  A part's slot is
// its item's ordinal + its CTA's: walking through the list, each next part raises one of
// the two, so that no two parts share one.
struct CacheList {
  long long items, slots;  // at most
  int grid;
  size_t head, ml, part;  // byte offsets
};
struct CacheShape {
  bool apart;      // prefixes are a list of their own (`pre`); else one list holds all
  CacheList list;  // the own keys' (and the prefixes')
  CacheList pre;
  size_t total;    // bytes
};
// A prefix's tiles of `rows` rows: those of its sequences' rows, and one a group for the
// remainders at most.
inline CacheShape cache_shape(long long B, long long Hkv, long long rows, int dv, bool quantised, long long capacity,
                              long long groups, long long prefix_capacity, int sms) {
  CacheShape s;
  s.apart = prefix_apart(groups, rows * B);
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  auto lay = [&](CacheList* l, long long entries, long long tiles, long long chunks, int item_rows, int min_chunks, long long ctas) {
    l->items = Hkv * tiles;
    const long long want = (Hkv * chunks + min_chunks - 1) / min_chunks;
    l->grid = (int)(want < 1 ? 1 : want < ctas ? want : ctas);
    l->slots = l->items + l->grid;
    l->head = take((size_t)(entries + 1) * sizeof(CacheHead));
    l->ml = take((size_t)l->slots * item_rows * 2 * sizeof(float));
    l->part = take((size_t)l->slots * item_rows * dv * sizeof(float));
  };
  const long long kc = cache_chunk_keys(quantised), own_tiles = B * ((rows + kCacheRows - 1) / kCacheRows);
  const long long pre_tiles = groups ? groups + rows * B / (s.apart ? kPrefixRows : kCacheRows) : 0;
  const long long own = own_tiles * ((capacity + kc - 1) / kc);
  if (s.apart) {
    lay(&s.list, B, own_tiles, own, kCacheRows, kCacheMinChunks, (long long)kCacheCtasPerSm * sms);
    lay(&s.pre, groups, pre_tiles, pre_tiles * ((prefix_capacity + kPrefixKeys - 1) / kPrefixKeys), kPrefixRows, kPrefixMinChunks, sms);
  } else {
    lay(&s.list, groups + B, own_tiles + pre_tiles, own + pre_tiles * ((prefix_capacity + kc - 1) / kc), kCacheRows,
        kCacheMinChunks, (long long)kCacheCtasPerSm * sms);
    s.pre = s.list;
  }
  s.total = at;
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
  FA_WALK int tiles(int item_rows) const { return (rows + item_rows - 1) / item_rows; }
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
template <int KC, int ROWS>
struct CacheCursor {
  long long at;  // in the whole list
  int e, h, r, c;
  CacheEntry n;
  FA_WALK void advance(const CacheParams& p, bool groups_ok, int k) {
    at += k;
    c += k;
    while (c >= n.chunks) {
      c -= n.chunks;
      if (++r < n.tiles(ROWS)) continue;
      r = 0;
      if (++h < p.Hkv) continue;
      h = 0;
      do {
        if (++e >= p.entries) {  // the list's end: stay there
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
struct CacheSlots {
  long long slot;
  int n, row;  // parts, row within the tile
};
FA_WALK CacheSlots cache_slots(const CacheHead& e, int rows, int item_rows, int h, int row, long long per) {
  CacheSlots l = {0, 0, row % item_rows};
  if (e.chunks == 0) return l;
  const int o = h * ((rows + item_rows - 1) / item_rows) + row / item_rows;
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
// The CTA's share [begin, end) of the list, and its first place.  CTA 0 also writes
// where each entry begins, for the join.
template <int KC, int ROWS>
struct CacheShare {
  long long begin, end;
  CacheCursor<KC, ROWS> start;
  int item;  // ordinal of the first place's item
};

template <int KC, int ROWS, int THREADS>
__device__ __forceinline__ CacheShare<KC, ROWS> cache_share(const CacheParams& p, bool groups_ok) {
  constexpr int WARPS = THREADS / 32;
  __shared__ long long s_work[WARPS], s_found_work;
  __shared__ int s_item[WARPS], s_found_e, s_found_item;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, entries = p.entries;
  long long total = 0;
  for (int e = threadIdx.x; e < entries; e += THREADS) {
    const CacheEntry n = cache_entry<KC>(p, e, groups_ok);
    total += (long long)p.Hkv * n.tiles(ROWS) * n.chunks;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
  if (lane == 0) s_work[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) total += s_work[w];
  __syncthreads();
  CacheShare<KC, ROWS> s;
  long long per = (total + gridDim.x - 1) / gridDim.x;
  per = per < p.min_chunks ? p.min_chunks : per;
  s.begin = per * blockIdx.x;
  s.end = s.begin + per < total ? s.begin + per : total;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.parts.head[entries].work = per;
    bool bad = !groups_ok;
    for (int e = 0; e < p.S && !bad; ++e) bad = __ldg(p.p_lengths + e) > (p.p_cols << p.page_log2);
    if (bad) cache_bad(p.status);
  }
  if (s.begin >= s.end && blockIdx.x) return s;
  long long base = 0;
  int item = 0;
  for (int e0 = 0; e0 < entries; e0 += THREADS) {
    const int e = e0 + threadIdx.x;
    long long work = 0;
    int items = 0;
    CacheEntry n = {};
    if (e < entries) {
      n = cache_entry<KC>(p, e, groups_ok);
      items = p.Hkv * n.tiles(ROWS);
      work = (long long)items * n.chunks;
      if (blockIdx.x == 0 && e >= p.S && __ldg(p.lengths + e - p.S) > (p.cols << p.page_log2)) cache_bad(p.status);
    }
    long long w = work;
    int i = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long wo = __shfl_up_sync(~0u, w, o);
      const int io = __shfl_up_sync(~0u, i, o);
      if (lane >= o) w += wo, i += io;
    }
    if (lane == 31) s_work[warp] = w, s_item[warp] = i;
    __syncthreads();
    long long all = 0;
    int all_items = 0;
#pragma unroll
    for (int v = 0; v < WARPS; ++v) {
      if (v < warp) w += s_work[v], i += s_item[v];
      all += s_work[v];
      all_items += s_item[v];
    }
    w += base - work;
    i += item - items;
    if (blockIdx.x == 0 && e < entries) p.parts.head[e] = {w, i, n.chunks};
    if (work && w <= s.begin && s.begin < w + work) s_found_e = e, s_found_work = w, s_found_item = i;
    base += all;
    item += all_items;
    __syncthreads();
    if (blockIdx.x && s.begin < base) break;
  }
  if (s.begin >= s.end) return s;
  CacheCursor<KC, ROWS>& c = s.start;
  c.e = s_found_e;
  c.n = cache_entry<KC>(p, c.e, groups_ok);
  const long long in = s.begin - s_found_work;
  const int o = (int)(in / c.n.chunks), tiles = c.n.tiles(ROWS);
  c.at = s.begin;
  c.c = (int)(in - (long long)o * c.n.chunks);
  c.h = o / tiles;
  c.r = o - c.h * tiles;
  s.item = s_found_item + o;
  return s;
}

// Position (counted within the own keys) of row t of sequence b; the row's sequence and
// head for row `row` of an item.
struct CacheRow {
  int b, g, t;
  bool valid;
};
__device__ __forceinline__ CacheRow cache_row(const CacheParams& p, const CacheEntry& n, int row) {
  CacheRow r;
  r.valid = row < n.rows;
  if (!r.valid) row = 0;
  const int per = p.G * p.T, s = row / per, left = row - s * per;
  r.b = n.first + s;
  r.g = left / p.T;
  r.t = left - r.g * p.T;
  return r;
}
#endif

}  // namespace fa
