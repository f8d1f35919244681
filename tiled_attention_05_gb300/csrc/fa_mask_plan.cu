// Mask plan: from document ids and prefix lengths to the intervals and tile
// ranges that the score-modified kernels walk.
//
//   row i (of Tq) sees keys [lo_i, hi_i) of Tk:
//     hi_i = min(end of its document, max(i + off + 1, prefix))   (causal; else Tk)
//     lo_i = max(start of its document, i + off - window + 1)     (window; else 0)
//   with off = Tk - Tq.  Where the key documents are in ascending order a
//   document is one run of keys and both ends come from binary searches.
//   Otherwise (flag by_key) the interval leaves the documents out and the
//   kernels compare them key by key, within the hull of the tiles that can hold
//   the row's document.
//   key j is seen by rows [first i with hi_i > j, first i with lo_i > j) where lo
//   and hi ascend in i; otherwise (flag by_row, and always with by_key) the
//   backward looks every row's interval up.  A row that sees nothing gets an
//   empty interval in its place of the order; the backward gives such a row no
//   weight anyway (its L is -inf).
//
// Small and bound by latency, of which the first fetch of its instructions is a
// large part: a cluster of 8 CTAs per batch entry, three phases over keys, rows
// and keys again with cluster barriers between them (0.3 us each), and as little
// code as will do.  T 8192: 24 us with each row's searches one after the other in
// global memory, 16.3 with four rows' side by side, unrolled, 14.4 rolled, 12.3 in
// shared memory; T 777, B 2: 9.
#include <climits>
#include <cooperative_groups.h>
#include <cstdint>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 1024;
constexpr int kGroup = kThreads / fa::kTile;  // tiles a CTA takes at a time
constexpr int kCtas = fa::kPlanCtas;
constexpr int kMaxSmem = 200 << 10;
constexpr int kNoKeyDoc = INT_MAX, kNoRowDoc = -1;  // unlike each other and every document
constexpr int T = fa::kTile;

struct PlanParams {
  fa::MaskInputs in;
  int *row_lo, *row_hi, *q_doc, *k_doc, *kv_beg, *kv_end, *key_from, *key_to, *m_beg, *m_end, *tile_doc_lo,
      *tile_doc_hi, *pair_order, *key_order, *by_key, *by_row;
  int Tq, Tk, q_tiles, kv_tiles, causal, window, prefix_per_row;
  int room;  // ints of dynamic shared memory
};

__device__ __forceinline__ bool is_doc(int id) { return id >= 0 && id != INT_MAX; }

// How many entries of the ascending arrays a0, a1 (n each) are <= v0, v1.
__device__ __noinline__ int2 search(const int* a0, const int* a1, int n, int v0, int v1) {
  int c0 = 0, c1 = 0;
#pragma unroll 1
  for (int step = n > 0 ? 1 << (31 - __clz(n)) : 0; step > 0; step >>= 1) {
    if (c0 + step <= n && a0[c0 + step - 1] <= v0) c0 += step;
    if (c1 + step <= n && a1[c1 + step - 1] <= v1) c1 += step;
  }
  return make_int2(c0, c1);
}

// An array of n entries as the search reads it: copied to shared memory where it
// fits (`room` entries), since every step of a search in global memory is a miss
// of ~0.3 us.
__device__ __forceinline__ const int* staged(const int* a, int n, int* buf, int room) {
  if (n > room) return a;
  for (int k = threadIdx.x; k < n; k += kThreads) buf[k] = a[k];
  return buf;
}

__device__ __forceinline__ bool any_flag(const int* flags) {
  int any = 0;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) any |= flags[c];
  return any != 0;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) fa_mask_plan_kernel(const PlanParams p) {
  extern __shared__ int buf[];
  fa_ptx::grid_next();
  fa_ptx::grid_previous();
  cg::cluster_group cluster = cg::this_cluster();
  const int b = blockIdx.x / kCtas, cta = blockIdx.x % kCtas;
  const int lane = threadIdx.x & 31;
  const int warp = cta * (kThreads / 32) + (threadIdx.x >> 5), warps = kCtas * (kThreads / 32);
  const long long qp = (long long)b * p.q_tiles * T, kp = (long long)b * p.kv_tiles * T;  // padded rows / keys before
  int* k_doc = p.k_doc + kp;
  int* row_lo = p.row_lo + qp;
  int* row_hi = p.row_hi + qp;
  const int* doc_k = p.in.doc_k ? p.in.doc_k + (long long)b * p.Tk : nullptr;
  const int* doc_q = p.in.doc_q ? p.in.doc_q + (long long)b * p.Tq : nullptr;
  const int off = p.Tk - p.Tq;

  // ---- keys: documents without the padding's ids, their order, each tile's span
  int bad = 0;
#pragma unroll 1
  for (int n = warp; n < p.kv_tiles; n += warps) {
    int lo = INT_MAX, hi = -1;
    bool none = false;
#pragma unroll 1
    for (int e = 0; e < T / 32; ++e) {
      const int j = n * T + e * 32 + lane;
      int d = kNoKeyDoc;
      if (j < p.Tk) {
        d = doc_k ? (is_doc(doc_k[j]) ? doc_k[j] : kNoKeyDoc) : 0;
        if (doc_k && j > 0) bad |= (is_doc(doc_k[j - 1]) ? doc_k[j - 1] : kNoKeyDoc) > d;
      }
      k_doc[j] = d;
      if (d != kNoKeyDoc) {
        lo = min(lo, d);
        hi = max(hi, d);
      } else {
        none = true;
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    // a tile with padding in it is not all one document: keep its ends apart
    if (__any_sync(0xffffffffu, none) && lo == hi) --lo;
    if (lane == 0) {
      p.tile_doc_lo[(long long)b * p.kv_tiles + n] = lo;
      p.tile_doc_hi[(long long)b * p.kv_tiles + n] = hi;
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) p.by_key[b * kCtas + cta] = bad;
  cluster.sync();

  // ---- rows: intervals, and the key tiles of each query tile (one row a thread)
  __shared__ int w_beg[kThreads / 32], w_end[kThreads / 32], w_dmin[kThreads / 32], w_dmax[kThreads / 32];
  const bool by_key = any_flag(p.by_key + b * kCtas);
  const int* sorted = doc_q && !by_key ? staged(k_doc, p.Tk, buf, p.room) : k_doc;
  __syncthreads();
#pragma unroll 1
  for (int m0 = cta * kGroup; m0 < p.q_tiles; m0 += kCtas * kGroup) {
    const int i = m0 * T + threadIdx.x, wid = threadIdx.x >> 5;
    int lo = p.Tk, hi = p.Tk, d = kNoRowDoc;  // rows past the last: empty, last in order
    if (i < p.Tq) {
      const int id = doc_q ? doc_q[i] : 0;
      const bool has = is_doc(id);
      lo = 0;
      hi = by_key && !has ? 0 : p.Tk;
      if (doc_q && !by_key) {  // (padding rows: both ends where the keys' padding starts)
        const int v = has ? id : kNoKeyDoc - 1;
        const int2 ends = search(sorted, sorted, p.Tk, has ? v - 1 : v, v);
        lo = ends.x;
        hi = ends.y;
      }
      if (has) d = id;
      if (p.causal) {
        int seen = i + off + 1;
        if (p.in.prefix) seen = max(seen, p.in.prefix[p.prefix_per_row ? (long long)b * p.Tq + i : (long long)b]);
        hi = min(hi, max(seen, 0));
      }
      if (p.window) lo = max(lo, min(i + off - p.window + 1, p.Tk));
      hi = max(hi, lo);
    }
    if (i < p.q_tiles * T) {
      row_lo[i] = lo;
      row_hi[i] = hi;
      p.q_doc[qp + i] = d;
    }
    const bool sees = lo < hi;
    const int beg = __reduce_min_sync(0xffffffffu, sees ? lo : INT_MAX), end = __reduce_max_sync(0xffffffffu, sees ? hi : 0);
    const int dmin = __reduce_min_sync(0xffffffffu, sees ? d : INT_MAX), dmax = __reduce_max_sync(0xffffffffu, sees ? d : -1);
    if (lane == 0) {
      w_beg[wid] = beg;
      w_end[wid] = end;
      w_dmin[wid] = dmin;
      w_dmax[wid] = dmax;
    }
    __syncthreads();
    const int m = m0 + wid;
    if (wid < kGroup && m < p.q_tiles) {  // one warp a tile
      const int from = wid * (T / 32) + lane % (T / 32);
      const int tbeg = __reduce_min_sync(0xffffffffu, w_beg[from]), tend = __reduce_max_sync(0xffffffffu, w_end[from]);
      int tb = 0, te = 0;
      if (tbeg < tend) {
        tb = tbeg / T;
        te = (tend + T - 1) / T;
        if (by_key) {  // only as far as tiles that can hold the rows' documents
          const int tmin = __reduce_min_sync(0xffffffffu, w_dmin[from]), tmax = __reduce_max_sync(0xffffffffu, w_dmax[from]);
          int first = INT_MAX, last = -1;
#pragma unroll 1
          for (int n = tb + lane; n < te; n += 32) {
            const long long at = (long long)b * p.kv_tiles + n;
            if (p.tile_doc_lo[at] <= tmax && p.tile_doc_hi[at] >= tmin) {
              first = min(first, n);
              last = max(last, n);
            }
          }
          tb = __reduce_min_sync(0xffffffffu, first);
          te = __reduce_max_sync(0xffffffffu, last) + 1;
          if (te == 0) tb = 0;
        }
      }
      if (lane == 0) {
        p.kv_beg[(long long)b * p.q_tiles + m] = tb;
        p.kv_end[(long long)b * p.q_tiles + m] = te;
      }
    }
    __syncthreads();
  }
  cluster.sync();

  // ---- keys again: the rows that see each, and the query tiles of each key tile
  bad = by_key;
  const int* his = staged(row_hi, p.Tq, buf, p.room / 2);
  const int* los = staged(row_lo, p.Tq, buf + p.room / 2, p.room / 2);
  __syncthreads();
#pragma unroll 1
  for (int t = cta * kThreads + threadIdx.x; t < max(p.Tq, p.kv_tiles * T); t += kCtas * kThreads) {
    if (t > 0 && t < p.Tq) bad |= los[t] < los[t - 1] || his[t] < his[t - 1];
    if (t < p.kv_tiles * T) {
      int2 rows = make_int2(1 << 30, 0);
      if (t < p.Tk) rows = search(his, los, p.Tq, t, t);
      p.key_from[kp + t] = rows.x;
      p.key_to[kp + t] = rows.y;
    }
  }
  // pairs of query tiles by work (a step with both tiles costs 1.5 of one with a
  // single tile): one warp a pair, which counts those before it
  const int pairs = (p.q_tiles + 1) / 2;
  const int *kv_beg = p.kv_beg + (long long)b * p.q_tiles, *kv_end = p.kv_end + (long long)b * p.q_tiles;
  auto work = [&](int y) {
    const int a = kv_end[2 * y] - kv_beg[2 * y], c = 2 * y + 1 < p.q_tiles ? kv_end[2 * y + 1] - kv_beg[2 * y + 1] : 0;
    return 2 * max(a, c) + min(a, c);
  };
#pragma unroll 1
  for (int y = warp; y < pairs; y += warps) {
    const int w = work(y);
    int before = 0;
#pragma unroll 1
    for (int z = lane; z < pairs; z += 32) {
      const int v = work(z);
      before += v > w || (v == w && z > y);  // (equal work: the later rows first)
    }
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) p.pair_order[(long long)b * pairs + before] = y;
  }
#pragma unroll 1
  for (int n = warp; n < p.kv_tiles; n += warps) {
    int first = INT_MAX, last = -1;
#pragma unroll 1
    for (int m = lane; m < p.q_tiles; m += 32) {
      const long long at = (long long)b * p.q_tiles + m;
      if (p.kv_beg[at] <= n && n < p.kv_end[at]) {
        first = min(first, m);
        last = max(last, m);
      }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) {
      p.m_beg[(long long)b * p.kv_tiles + n] = last >= 0 ? first : 0;
      p.m_end[(long long)b * p.kv_tiles + n] = last + 1;
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) p.by_row[b * kCtas + cta] = bad;
  cluster.sync();

  // ---- key tiles by work
  const int *m_beg = p.m_beg + (long long)b * p.kv_tiles, *m_end = p.m_end + (long long)b * p.kv_tiles;
#pragma unroll 1
  for (int n = warp; n < p.kv_tiles; n += warps) {
    const int w = m_end[n] - m_beg[n];
    int before = 0;
#pragma unroll 1
    for (int z = lane; z < p.kv_tiles; z += 32) {
      const int v = m_end[z] - m_beg[z];
      before += v > w || (v == w && z < n);
    }
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) p.key_order[(long long)b * p.kv_tiles + before] = n;
  }
}

}  // namespace

namespace fa {

cudaError_t launch_mask_plan(const Problem& pr, const MaskInputs& in, void* plan, cudaStream_t stream) {
  if (pr.B == 0) return cudaSuccess;
  const PlanLayout l = plan_layout(pr);
  int* a = static_cast<int*>(plan);
  PlanParams p;
  p.in = in;
  p.row_lo = a + l.row_lo;
  p.row_hi = a + l.row_hi;
  p.q_doc = a + l.q_doc;
  p.k_doc = a + l.k_doc;
  p.kv_beg = a + l.kv_beg;
  p.kv_end = a + l.kv_end;
  p.key_from = a + l.key_from;
  p.key_to = a + l.key_to;
  p.m_beg = a + l.m_beg;
  p.m_end = a + l.m_end;
  p.tile_doc_lo = a + l.tile_doc_lo;
  p.tile_doc_hi = a + l.tile_doc_hi;
  p.pair_order = a + l.pair_order;
  p.key_order = a + l.key_order;
  p.by_key = a + l.by_key;
  p.by_row = a + l.by_row;
  p.Tq = pr.Tq;
  p.Tk = pr.Tk;
  p.q_tiles = pr.q_tiles();
  p.kv_tiles = pr.kv_tiles();
  p.causal = pr.causal;
  p.window = pr.window;
  p.prefix_per_row = in.prefix_per_row;
  // room for the keys' documents, then for the rows' two ends
  const long long want = 4 * (pr.Tk > 2LL * pr.Tq ? (long long)pr.Tk : 2LL * pr.Tq);
  const int smem = (int)(want < kMaxSmem ? want : kMaxSmem);
  p.room = smem / 4;
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(fa_mask_plan_kernel), kMaxSmem);
  if (e != cudaSuccess) return e;
  return launch_next(fa_mask_plan_kernel, (unsigned)pr.B * kCtas, kThreads, smem, stream, p);
}

}  // namespace fa
