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
// CTAs an SM.  e4m3 takes about twice the instructions a byte (its codes become fp16), so
// it needs the warps.
constexpr int cache_ctas(bool quantised, bool few) { return quantised ? 3 : 2; }
constexpr bool cache_few(long long rows, bool prefixes) { return rows <= 8 && !prefixes; }
// A CTA gets this much work at least, in chunks of keys, and an item counts as so many
// chunks more than it has, for its set-up and the joining of its parts: 16 where there are two
// tiles of 8 rows, which are joined one after the other (4 rows each of 48 sequences, 16 / 4 heads,
// e4m3, at 8, 12, 16, 24: 50, 46, 41.5, 43 us; 16 / 8 heads of 64, one row each of 128, beside
// prefixes, at 8, 16, 24: 48.2, 48.5, 54.2).
constexpr int kCacheMinChunks = 8;
constexpr int cache_item(bool few) { return few ? 8 : 16; }
// Where no item can have more chunks than this (and there are no prefixes), a CTA takes its
// items whole: those that begin in its share.  What can be is what the tables hold, which the
// host knows, not the lengths: a table kept for the longest answer is not among these.  Then
// there are no parts, no workspace and no join.  (On the GPU, whole / in parts, us, heads of 128,
// bf16: 1 sequence of 100, 256, 500 keys 5.7 / 7.2, 7.1 / 7.1, 9.7 / 7.4; 64 of 100, 256, 500
// 10.2 / 12.6, 13.0 / 15.2, 26.1 / 25.4; on the host it is one launch and allocation less, 6 us.)
constexpr int kCacheWhole = 16;
// Prefixes of many rows have a list of their own (fa_cache_prefix_kernel), with items of
// two tiles of 128 rows and chunks of 128 keys.
constexpr int kPrefixRows = 256, kPrefixKeys = 128, kPrefixMinChunks = 4, kPrefixItem = 2;

struct CacheHead {
  int work;    // work of all entries before this one
  int item;    // items of all entries before this one
  int chunks;  // of one item of this entry
};
// Division of numbers below 2^30 by a positive one, by its reciprocal (one short at most).
struct Divide {
  unsigned by, inverse;
  static Divide of(int by) { return {(unsigned)by, by == 1 ? 0xffffffffu : (unsigned)((1ull << 32) / (unsigned)by)}; }
  FA_WALK int operator()(int n) const {
#ifdef __CUDA_ARCH__
    unsigned q = __umulhi((unsigned)n, inverse);
#else
    unsigned q = (unsigned)(((unsigned long long)(unsigned)n * inverse) >> 32);
#endif
    return (int)(q + ((q + 1) * by <= (unsigned)n));
  }
};
// Parts of items (of `rows` rows each) that a join adds up.
struct CacheParts {
  CacheHead* head;  // [entries + 1]; the last one's work: a CTA's share; its item: the bundle
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
  // Prefixes of many rows and the own keys run side by side, on SMs of their own: the two
  // kernels divide `sms` between them by their work (0: a kernel has all).
  int sms, groups;  // groups: S, also for the kernel of the own keys (whose S is 0)
  int chunk_cost;   // of a chunk of own keys; of a prefix's 1024
  int per_sm;       // CTAs of the own keys' kernel on an SM
  int own_item;    // what an item of the own keys' list counts (cache_item)
  int joined;      // whole items too leave their part for the join
  int whole;       // items are not split (kCacheWhole)
  Divide by_T, by_GT;  // rows of a head, of a sequence
  int max_items;   // that the workspace has slots for
  int* look;       // [CTAs] prefixes in bf16 with a window: whether the results hold a NaN or an infinity
  int capped, min_chunks;
  float scale_log2;
  CapParams cap;
};
// A prefix of several tiles of rows, the only one of a call, is walked by so many CTAs side
// by side, each with a tile of its own: they meet the same keys at about the same time, and
// HBM gives them once (walked one after the other, 1024 rows over 32768 keys of bf16 read
// 402 MB where there are 134).  1: each CTA walks all of an entry's tiles.
FA_WALK int cache_bundle(int groups, int tiles, int ctas) { return groups == 1 && tiles > 1 && tiles <= ctas ? tiles : 1; }

// What the join adds to the own keys' parts: those of the prefixes.
struct CacheJoin {
  CacheParams p;       // p.S = 0: no prefixes; parts: of the own keys
  int own;             // entry of sequence 0 in its list
  int own_entries;     // of that list
  CacheParts pre;      // parts of the prefixes, in items of pre_rows rows
  int pre_rows, pre_entries;
  Divide by_Hq, by_G;
};

// The kernels, by the type of the cache, and the join of their parts.
cudaError_t launch_cache_attn_e4m3(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream);
cudaError_t launch_cache_attn_bf16(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream);
cudaError_t launch_cache_prefix_e4m3(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream);
cudaError_t launch_cache_prefix_bf16(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream);
// bf16 with a window: the kernel, and after it, for the shares that it marked in `look`, again.
cudaError_t launch_cache_prefix_window(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream);
cudaError_t launch_cache_prefix_careful(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream);
cudaError_t launch_cache_join(const CacheJoin& j, int dv, cudaStream_t stream);

// Keys of a chunk, the unit of the walk: what one warp holds in one stage of its ring.
constexpr int kCacheKeys = 16;

// What an SM takes for a chunk of own keys (its bytes at ~90 a ns) over a prefix's two tiles
// of 128 keys (1.5 us at heads of 128; in e4m3 they take longer, and the own keys' rate that
// divides best is higher), in 1024ths.  One rate for each type, whatever the items' lengths: the
// own keys' own rate falls where those are short.  (64 answers to 8192 tokens, e4m3, at 80, 100,
// 110, 130, 170 a ns: 49, 47, 43, 43, 49 us; 256 to 32768, bf16, at 70, 80, 90, 100: 165, 164, 165, 178.)
constexpr int cache_chunk_cost(int d, int dv, bool quantised) {
  return quantised ? kCacheKeys * (d + dv + 8) * 1024 / (110 * 1500) * 256 / (d + dv)
                   : kCacheKeys * 2 * 256 * 1024 / (90 * 1500);
}
// Whether the prefixes go through the kernel that takes 128 rows at a time (`rows`: those
// of all sequences' kv heads): from so many rows a group on, as the decode kernel reads a
// prefix's keys, out of L2, once for each 16 rows, and spends as many instructions on a key
// of 64 channels as on one of 128, and e4m3 costs the other kernel a conversion.  (Decode kernel / apart, us,
// at that number of rows: bf16, heads of 128, 32 rows a group: 8 groups of 4000 keys 40 / 42, one of 40000 53 / 60;
// 48 rows: 4 of 4000 50 / 46; heads of 64, 32 rows, slopes, 8 of 2001 51 / 48.  e4m3, 32 rows: one of 40000 46 / 81;
// 64 rows: 4 of 4000 51 / 53, 8 of 2001 with heads of 64 67 / 81; 96: 8 of 2000 81 / 71.)
inline bool prefix_apart(long long groups, long long rows, bool quantised, int dv) {
  return groups > 0 && rows > (quantised ? 64 : dv == 64 ? 16 : 32) * groups;
}

// Slots of the workspace and CTAs of a call, from what the host knows.  A part's slot is
// its item's ordinal + its CTA's (both of bundles, times the bundle, + the tile): walking through the list, each next part raises one of
// the two, so that no two parts share one.
struct CacheList {
  long long items, slots;  // at most
  int grid;
  size_t head, ml, part;  // byte offsets
};
struct CacheShape {
  bool fits;       // items and chunks can be counted in 32 bits
  bool whole;      // no item is split: no workspace
  bool apart;      // prefixes are a list of their own (`pre`); else one list holds all
  CacheList list;  // the own keys' (and the prefixes')
  CacheList pre;
  size_t look;     // byte offset
  size_t total;    // bytes
};
// A prefix's tiles of `rows` rows: those of its sequences' rows, and one a group for the
// remainders at most.
inline CacheShape cache_shape(long long B, long long Hkv, long long rows, int dv, bool quantised, long long capacity,
                              long long groups, long long prefix_capacity, int sms) {
  CacheShape s;
  s.apart = prefix_apart(groups, rows * B, quantised, dv);
  s.whole = groups == 0 && capacity <= kCacheWhole * kCacheKeys;
  s.fits = true;
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  auto lay = [&](CacheList* l, long long entries, long long tiles, double chunks, int item_rows, int min_chunks, int item, long long ctas) {
    l->items = Hkv * tiles;
    chunks += (double)tiles * item;
    s.fits = s.fits && l->items <= (1 << 30) && Hkv * (double)chunks < (double)(1 << 30);
    const double want = Hkv * chunks / min_chunks + 1;
    l->grid = (int)(want < ctas ? want : ctas);
    l->slots = l->items + l->grid;
    l->head = take((size_t)(entries + 1) * sizeof(CacheHead));
    l->ml = take((size_t)l->slots * item_rows * 2 * sizeof(float));
    l->part = take((size_t)l->slots * item_rows * dv * sizeof(float));
  };
  const long long kc = kCacheKeys, own_tiles = B * ((rows + kCacheRows - 1) / kCacheRows);
  const long long pre_tiles = groups ? groups + rows * B / (s.apart ? kPrefixRows : kCacheRows) : 0;
  const double own = (double)own_tiles * ((capacity + kc - 1) / kc);
  const bool few = cache_few(rows, groups && !s.apart);
  const long long ctas = (long long)sms * cache_ctas(quantised, few);
  if (s.apart) {
    lay(&s.list, B, own_tiles, own, kCacheRows, kCacheMinChunks, cache_item(few), ctas);
    lay(&s.pre, groups, pre_tiles, (double)pre_tiles * ((prefix_capacity + kPrefixKeys - 1) / kPrefixKeys), kPrefixRows, kPrefixMinChunks, kPrefixItem, sms);
  } else {
    lay(&s.list, groups + B, own_tiles + pre_tiles, own + (double)pre_tiles * ((prefix_capacity + kc - 1) / kc), kCacheRows,
        kCacheMinChunks, cache_item(few), ctas);
    s.pre = s.list;
  }
  s.look = take(s.apart && !quantised ? s.pre.grid * sizeof(int) : 0);
  s.total = s.whole ? 0 : at;
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
  int from;    // first key that any row sees
  int chunk0;  // its chunk
  int chunks;  // from there on
  FA_WALK int tiles(int item_rows) const { return (rows + item_rows - 1) / item_rows; }
};

FA_WALK int cache_length(const CacheParams& p, int b) {
  return cache_clamp(cache_ld(p.lengths + b), p.cols << p.page_log2);
}
// Sequences [first, end) of group s; none where the starts do not fit.
FA_WALK void cache_group(const CacheParams& p, int s, int* first, int* end) {
  *first = p.p_starts ? cache_ld(p.p_starts + s) : 0;
  *end = p.p_starts ? cache_ld(p.p_starts + s + 1) : p.B;
  if (*first < 0 || *end > p.B || *first > *end) *first = *end = 0;
}

// The least position among the own keys that a row has which sees anything, of sequence b and of
// sequences [first, end), group s; 2^31 - 1 where there is none.  With a window the first key
// of the prefix that any row sees hangs on it.
FA_WALK int cache_least_of(const CacheParams& p, int b) {
  const int n = cache_length(p, b);
  return n <= 0 ? 0x7fffffff : n > p.T ? n - p.T : 0;
}
#ifdef __CUDACC__
// A CTA works it out once for the first groups (cache_share); for those behind them whoever asks does.
constexpr int kCacheLeast = 32;
__device__ __forceinline__ int* cache_leasts() {
  __shared__ int least[kCacheLeast];
  return least;
}
#endif
FA_WALK int cache_least(const CacheParams& p, int s, int first, int end) {
#ifdef __CUDACC__
  if (s < kCacheLeast) return cache_leasts()[s];
#endif
  int least = 0x7fffffff;
#pragma unroll 1
  for (int b = first; b < end; ++b) {
    const int at = cache_least_of(p, b);
    least = at < least ? at : least;
  }
  return least;
}

FA_WALK void cache_span(CacheEntry* n, int first_key, int KC) {
  n->from = first_key > 0 ? first_key : 0;
  n->chunk0 = n->from / KC;
  n->chunks = n->rows > 0 && first_key < n->keys ? (n->keys + KC - 1) / KC - n->chunk0 : 0;
}
// WINDOW (here and below): the call may have one.  (Code that is jumped over costs a kernel's start
// too: 64 answers to 8192 tokens in e4m3 took 44.6 us with it, 43.2 without.)
template <int KC, bool WINDOW = true>
FA_WALK CacheEntry cache_prefix(const CacheParams& p, int s) {
  CacheEntry n;
  int end, first_key = 0;
  cache_group(p, s, &n.first, &end);
  n.rows = (end - n.first) * p.G * p.T;
  n.keys = cache_clamp(cache_ld(p.p_lengths + s), p.p_cols << p.page_log2);
  if (WINDOW && p.window) {
    const int least = cache_least(p, s, n.first, end);
    first_key = least == 0x7fffffff ? n.keys : n.keys - p.window + 1 + least;  // (both lengths are 2^30 at most)
  }
  cache_span(&n, first_key, KC);
  return n;
}
template <int KC>
FA_WALK CacheEntry cache_own(const CacheParams& p, int b) {
  CacheEntry n;
  n.first = b;
  n.rows = p.G * p.T;
  n.keys = cache_length(p, b);
  cache_span(&n, p.window ? (n.keys > p.T ? n.keys - p.T : 0) - p.window + 1 : 0, KC);
  return n;
}
template <int KC, bool WINDOW = true>
FA_WALK CacheEntry cache_entry(const CacheParams& p, int e) {
  return e < p.S ? cache_prefix<KC, WINDOW>(p, e) : cache_own<KC>(p, e - p.S);
}

// A place in the list: that of chunk c of the item of tile r, kv head h, entry e.  ITEM:
// what an item counts beside its chunks, behind them.
template <int KC, int ROWS, int ITEM, bool WINDOW = true>
struct CacheCursor {
  int at;  // in the whole list
  int e, h, r, c;
  int item;  // ordinal of the item (of a bundle's)
  int bundle;
  CacheEntry n;
  FA_WALK int tiles() const { return n.tiles(ROWS) / bundle; }
  FA_WALK int end(const CacheParams& p, int share_end) const {
    return p.whole || c + share_end - at >= n.chunks ? n.chunks : c + share_end - at;
  }
  FA_WALK void next(const CacheParams& p) {  // the next item's first chunk
    at += n.chunks + ITEM - c;
    c = 0;
    ++item;
    if (++r < tiles()) return;
    r = 0;
    if (++h < p.Hkv) return;
    h = 0;
    while (++e < p.entries) {
      n = cache_entry<KC, WINDOW>(p, e);
      if (n.chunks || p.whole) return;  // (whole: a row that sees nothing is written by its item)
      item += p.Hkv * tiles();
    }
    at = 0x3fffffff;  // the list's end
  }
  // To the share's start `in` units into entry e's items, the first of which is `first`.
  FA_WALK void start(const CacheParams& p, int side_by_side, int entry, int first, int begin, int in) {
    bundle = side_by_side;
    e = entry;
    n = cache_entry<KC, WINDOW>(p, e);
    const int o = in / (n.chunks + ITEM);
    at = begin;
    c = in - o * (n.chunks + ITEM);
    h = o / tiles();
    r = o - h * tiles();
    item = first + o;
    if (p.whole ? c > 0 : c >= n.chunks) next(p);
  }
};

// Where the join finds the parts of row `row` of an entry's kv head h: `n` slots from
// `slot` on (`per`: a CTA's share).
struct CacheSlots {
  long long slot;    // of the first part; the next ones are `step` apart
  int n, row, step;  // parts, row within the tile
};
FA_WALK CacheSlots cache_slots(const CacheHead& e, int rows, int item_rows, int item_work, int bundle, int h, int row, int per) {
  CacheSlots l = {0, 0, row % item_rows, bundle};
  if (e.chunks == 0) return l;
  const int tile = row / item_rows, o = h * ((rows + item_rows - 1) / item_rows / bundle) + tile / bundle;
  const int at = e.work + o * (e.chunks + item_work), c0 = at / per, c1 = (at + e.chunks - 1) / per;
  l.slot = ((long long)e.item + o + c0) * bundle + tile % bundle;
  l.n = c1 - c0 + 1;
  return l;
}

// CTA `cta`'s share of a list of `all` (below 2^30) cut for `ctas`; those from there on have
// nothing (their number times the share may pass 32 bits).  Returns the share's size.
FA_WALK int cache_cut(int all, unsigned ctas, int min_chunks, int cta, int* begin, int* end) {
  const int even = (int)(((unsigned)all + ctas - 1) / ctas), per = even > min_chunks ? even : min_chunks;
  const bool some = (unsigned)cta < ctas && (unsigned)per * (unsigned)cta < (unsigned)all;
  *begin = some ? per * cta : all;
  *end = all - *begin > per ? *begin + per : all;
  return per;
}

#ifdef __CUDACC__
// An index that does not fit: the device status word says so (a timeout stays).
__device__ __forceinline__ void cache_bad(int* status) { atomicCAS(status, 0, fa_ptx::DEV_BAD_TABLE); }

// The CTA's share [begin, end) of the list, and its first place.  CTA 0 also writes
// where each entry begins, for the join.  (Code that runs once is short rather than
// fast: an instruction that no CTA has run yet costs some 10 to 20 cycles.)
template <class Cursor>
struct CacheShare {
  int begin, end;
  int cta, tile;  // place among the bundles, tile within its own
  Cursor start;
};

template <int KC, int ROWS, int ITEM, int THREADS, bool WINDOW = true>
__device__ __forceinline__ CacheShare<CacheCursor<KC, ROWS, ITEM, WINDOW>> cache_share(const CacheParams& p) {
  constexpr int WARPS = THREADS / 32;
  __shared__ long long s_sum[WARPS][3];
  __shared__ int s_found[3];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr bool PRE = ROWS == kPrefixRows;
  const int groups = p.S > p.groups ? p.S : p.groups;
  if (WINDOW && p.window && groups) {
#pragma unroll 1
    for (int s = warp; s < min(groups, kCacheLeast); s += WARPS) {
      int first, end, least = 0x7fffffff;
      cache_group(p, s, &first, &end);
#pragma unroll 1
      for (int b = first + lane; b < end; b += 32) least = min(least, cache_least_of(p, b));
      least = __reduce_min_sync(~0u, least);
      if (lane == 0) cache_leasts()[s] = least;
    }
    __syncthreads();
  }
  // CTAs side by side (see cache_bundle); the other list's kernel has to know, too
  const int pre_tiles = (PRE || p.sms) && p.groups == 1 ? cache_prefix<kPrefixKeys, WINDOW>(p, 0).tiles(kPrefixRows) : 1;
  const int pre_bundle = cache_bundle(p.groups, pre_tiles, PRE ? (int)gridDim.x : p.sms), bundle = PRE ? pre_bundle : 1;
  const int each = (p.entries + THREADS - 1) / THREADS;
  const int e0 = min((int)threadIdx.x * each, p.entries), e1 = min(e0 + each, p.entries);
  long long sum[2] = {0, 0};  // work and items of this thread's entries
#pragma unroll 1
  for (int e = e0; e < e1; ++e) {
    const CacheEntry n = cache_entry<KC, WINDOW>(p, e);
    const int items = p.Hkv * (n.tiles(ROWS) / bundle);
    if (n.chunks || p.whole) sum[0] += (long long)items * (n.chunks + ITEM);
    sum[1] += items;
  }
  const long long mine = sum[0], my_items = sum[1];
  long long other = 0;  // work of the list that runs beside this one
  if (p.sms) {
#pragma unroll 1
    for (int e = threadIdx.x; e < (PRE ? p.B : p.groups); e += THREADS) {
      const CacheEntry n = PRE ? cache_own<kCacheKeys>(p, e) : cache_prefix<kPrefixKeys, WINDOW>(p, e);
      if (n.chunks) other += (long long)p.Hkv * n.tiles(PRE ? kCacheRows : kPrefixRows) * (n.chunks + (PRE ? p.own_item : kPrefixItem));
    }
  }
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(~0u, sum[0], o), b = __shfl_up_sync(~0u, sum[1], o);
    if (lane >= o) sum[0] += a, sum[1] += b;
    other += __shfl_xor_sync(~0u, other, o);
  }
  if (lane == 31) s_sum[warp][0] = sum[0], s_sum[warp][1] = sum[1], s_sum[warp][2] = other;
  __syncthreads();
  other = 0;
  long long total = 0, items = 0, base = sum[0] - mine, item = sum[1] - my_items;
#pragma unroll 4
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) base += s_sum[w][0], item += s_sum[w][1];
    total += s_sum[w][0];
    items += s_sum[w][1];
    other += s_sum[w][2];
  }
  // groups that overlap can ask for more than there is room for: then there is no work
  const bool room = items <= p.max_items && total < (1 << 30);
  CacheShare<CacheCursor<KC, ROWS, ITEM, WINDOW>> s;
  const int all = room ? (int)total : 0;
  unsigned ctas = gridDim.x;
  if (p.sms) {  // as many SMs as its part of the cost, one at least (the CTAs from there on have nothing)
    const float pre = 1024.f * (float)(PRE ? total * bundle : other), own = (float)p.chunk_cost * (float)(PRE ? other : total);
    int on_pre = own > 0.f ? min(max((int)((float)p.sms * pre / (pre + own) + 0.5f), 1), p.sms - 1) : p.sms;
    on_pre = max(on_pre - on_pre % pre_bundle, min(pre_bundle, p.sms));  // whole bundles, one at least
    ctas = min(ctas / bundle, (unsigned)(PRE ? on_pre / bundle : max(p.sms - on_pre, 1) * p.per_sm));
  }
  s.tile = (int)blockIdx.x % bundle;
  s.cta = (int)blockIdx.x / bundle;
  const int per = cache_cut(all, ctas, p.min_chunks, s.cta, &s.begin, &s.end);
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0 && !p.whole) p.parts.head[p.entries].work = per, p.parts.head[p.entries].item = bundle;
    bool bad = !room;
    int w = (int)base, i = (int)item;
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
      const CacheEntry n = cache_entry<KC, WINDOW>(p, e);
      const int own = p.Hkv * (n.tiles(ROWS) / bundle);
      if (!p.whole) p.parts.head[e] = {w, i, room ? n.chunks : 0};
      if (n.chunks) w += own * (n.chunks + ITEM);
      i += own;
      if (e < p.S) {  // (the runs are in order and disjoint)
        bad = bad || __ldg(p.p_lengths + e) > (p.p_cols << p.page_log2);
        if (p.p_starts) {
          const int a = __ldg(p.p_starts + e), z = __ldg(p.p_starts + e + 1);
          bad = bad || a < 0 || a > z || z > p.B;
        }
      } else {
        bad = bad || __ldg(p.lengths + e - p.S) > (p.cols << p.page_log2);
      }
    }
    if (bad) cache_bad(p.status);
  }
  if (base <= s.begin && s.begin < base + mine && room) {
    int e = e0, w = (int)base, i = (int)item;
#pragma unroll 1
    for (;; ++e) {
      const CacheEntry n = cache_entry<KC, WINDOW>(p, e);
      const int own = p.Hkv * (n.tiles(ROWS) / bundle);
      const int all = n.chunks || p.whole ? own * (n.chunks + ITEM) : 0;
      if (s.begin < w + all) break;
      w += all;
      i += own;
    }
    s_found[0] = e, s_found[1] = w, s_found[2] = i;
  }
  __syncthreads();
  if (s.begin >= s.end) return s;
  s.start.start(p, bundle, s_found[0], s_found[2], s.begin, s.begin - s_found[1]);
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
  const int s = p.by_GT(row), left = row - s * p.G * p.T;
  r.b = n.first + s;
  r.g = p.by_T(left);
  r.t = left - r.g * p.T;
  return r;
}
#endif

}  // namespace fa
