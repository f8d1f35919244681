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
// Small and bound by latency: a cluster of 8 CTAs per batch entry, three
// phases over keys, rows and keys again, with cluster barriers between them;
// the arrays stay in L2.
#include <climits>
#include <cooperative_groups.h>
#include <cstdint>

#include "fa_internal.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512;
constexpr int kCtas = fa::kPlanCtas;
constexpr int kNoKeyDoc = INT_MAX, kNoRowDoc = -1;  // unlike each other and every document
constexpr int T = fa::kTile;

struct PlanParams {
  fa::MaskInputs in;
  int *row_lo, *row_hi, *q_doc, *k_doc, *kv_beg, *kv_end, *key_from, *key_to, *m_beg, *m_end, *tile_doc_lo,
      *tile_doc_hi, *by_key, *by_row;
  int Tq, Tk, q_tiles, kv_tiles, causal, window, prefix_per_row;
};

__device__ __forceinline__ bool is_doc(int id) { return id >= 0 && id != INT_MAX; }

// First index in [0, n) with a[index] > v (upper) or >= v; n if there is none.
template <bool UPPER>
__device__ __forceinline__ int search(const int* a, int n, int v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (int)(((unsigned)lo + (unsigned)hi) >> 1);
    const int x = a[mid];
    if (UPPER ? x > v : x >= v)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ bool any_flag(const int* flags) {
  int any = 0;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) any |= flags[c];
  return any != 0;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) fa_mask_plan_kernel(const PlanParams p) {
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
  for (int n = warp; n < p.kv_tiles; n += warps) {
    int lo = INT_MAX, hi = -1;
    bool none = false;
#pragma unroll
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
  __threadfence();
  cluster.sync();

  // ---- rows: intervals, and the key tiles of each query tile
  const bool by_key = any_flag(p.by_key + b * kCtas);
  for (int m = warp; m < p.q_tiles; m += warps) {
    int beg = INT_MAX, end = 0, dmin = INT_MAX, dmax = -1;
#pragma unroll
    for (int e = 0; e < T / 32; ++e) {
      const int i = m * T + e * 32 + lane;
      int lo = p.Tk, hi = p.Tk, d = kNoRowDoc;  // rows past the last: empty, last in order
      if (i < p.Tq) {
        const int id = doc_q ? doc_q[i] : 0;
        const bool has = is_doc(id);
        if (has) d = id;
        lo = 0;
        hi = p.Tk;
        if (doc_q && !by_key) {
          lo = search<false>(k_doc, p.Tk, has ? id : kNoKeyDoc);
          hi = has ? search<true>(k_doc, p.Tk, id) : lo;
        } else if (!has) {
          hi = 0;
        }
        if (p.causal) {
          int seen = i + off + 1;
          if (p.in.prefix)
            seen = max(seen, p.in.prefix[p.prefix_per_row ? (long long)b * p.Tq + i : (long long)b]);
          hi = min(hi, max(seen, 0));
        }
        if (p.window) lo = max(lo, min(i + off - p.window + 1, p.Tk));
        hi = max(hi, lo);
        if (lo < hi) {
          beg = min(beg, lo);
          end = max(end, hi);
          dmin = min(dmin, d);
          dmax = max(dmax, d);
        }
      }
      row_lo[i] = lo;
      row_hi[i] = hi;
      p.q_doc[qp + i] = d;
    }
    beg = __reduce_min_sync(0xffffffffu, beg);
    end = __reduce_max_sync(0xffffffffu, end);
    int tb = 0, te = 0;
    if (beg < end) {
      tb = beg / T;
      te = (end + T - 1) / T;
      if (by_key) {  // only as far as tiles that can hold the rows' documents
        dmin = __reduce_min_sync(0xffffffffu, dmin);
        dmax = __reduce_max_sync(0xffffffffu, dmax);
        int first = INT_MAX, last = -1;
        for (int n = tb + lane; n < te; n += 32) {
          const long long at = (long long)b * p.kv_tiles + n;
          if (p.tile_doc_lo[at] <= dmax && p.tile_doc_hi[at] >= dmin) {
            first = min(first, n);
            last = max(last, n);
          }
        }
        first = __reduce_min_sync(0xffffffffu, first);
        last = __reduce_max_sync(0xffffffffu, last);
        tb = last >= 0 ? first : 0;
        te = last + 1;
      }
    }
    if (lane == 0) {
      p.kv_beg[(long long)b * p.q_tiles + m] = tb;
      p.kv_end[(long long)b * p.q_tiles + m] = te;
    }
  }
  __threadfence();
  cluster.sync();

  // ---- keys again: the rows that see each, and the query tiles of each key tile
  bad = by_key;
  for (int i = cta * kThreads + threadIdx.x; i < p.Tq; i += kCtas * kThreads)
    if (i > 0) bad |= row_lo[i] < row_lo[i - 1] || row_hi[i] < row_hi[i - 1];
  for (int n = warp; n < p.kv_tiles; n += warps) {
#pragma unroll
    for (int e = 0; e < T / 32; ++e) {
      const int j = n * T + e * 32 + lane;
      int from = 1 << 30, to = 0;
      if (j < p.Tk) {
        from = search<true>(row_hi, p.Tq, j);
        to = search<true>(row_lo, p.Tq, j);
      }
      p.key_from[kp + j] = from;
      p.key_to[kp + j] = to;
    }
    int first = INT_MAX, last = -1;
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
  p.by_key = a + l.by_key;
  p.by_row = a + l.by_row;
  p.Tq = pr.Tq;
  p.Tk = pr.Tk;
  p.q_tiles = pr.q_tiles();
  p.kv_tiles = pr.kv_tiles();
  p.causal = pr.causal;
  p.window = pr.window;
  p.prefix_per_row = in.prefix_per_row;
  fa_mask_plan_kernel<<<(unsigned)pr.B * kCtas, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
