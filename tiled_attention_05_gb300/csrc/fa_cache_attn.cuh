// Attention of the newest tokens over a paged key/value cache (fa_cache_attention).
//
//   O = softmax(scale q K^T, modified and masked) V,  L = logsumexp
// for a few rows per sequence.  Every key and value byte is read once and takes few
// operations, so HBM bounds it; the kernel's work is to keep enough loads in flight.
// Measured, 32 / 8 heads of 128, one row each: 4 x 50000 to 65536 keys in bf16, 146 us (6.7 TB/s);
// 32 x 8192 in e4m3, 91 us (6.1 TB/s; its start of 3 to 4 us is the rest); 4 rows each of
// 48 x 3 to 7000, capped, 16 / 4 heads, 38 us (3.8 TB/s: items of 1 to 4 us have their
// starts and ends beside them).
//
// Split.  The keys of all items (sequence or shared prefix, kv head, tile of 16 rows)
// form one list of chunks of 16 keys, cut into equal shares, one
// for each CTA, whatever the lengths are.  A share that begins or ends inside an item
// leaves that item's part (unnormalised O, its reference and sum, in fp32) in the
// workspace, and a second kernel joins the parts in their order.  A prefix's rows are those
// of all its sequences; where they are many it goes through fa_cache_prefix.cuh.
//
// Warps.  Each of the CTA's four takes every fourth chunk of the share, through a ring
// of its own in shared memory (cp.async, no barrier between warps), and carries its own
// running maximum, sum and O.  The loads run ahead over the items' borders.  At an
// item's end the four are added up through shared memory.
//
// Products (mma.m16n8k16, fp32 accumulators; at these rows and bytes they take a
// fraction of the time that HBM does).  Keys and channels are the 16 rows of the left
// operand, the query rows the 8 columns, so that nothing of a tile is idle:
//   S^T = K Q^T, 16 keys x 8 rows;  O^T += V^T P^T, 16 channels x 8 rows a tile.
// What a quad's lane i holds of a key or value is 16-byte pieces i, i + 4, ... of its row:
// the channels are dealt to the k slots, and to O's rows, to suit that.  The pieces are
// swizzled in shared memory so that both reads are free of conflicts.  The weights come
// out as P^T's transpose, which movmatrix turns over.  Two tiles of rows share the
// operands made of keys and values.  (With the query rows as the 16 rows, half idle or more, and
// each code turned into the right operand: 106 us for 95, call and join, of 32 x 8192.)
//
// e4m3 rows carry an fp32 scale.  Codes become fp16 exactly; q is brought to fp16 by its
// row's power of two (bf16's 8 bits fit into fp16's 11; what is 2^-24 of the row's
// largest value is lost).  The key's scale multiplies the score.  The value's goes into
// the exponent, t = score + log2(v_scale), and the softmax's reference follows the
// maximum of t: the weights w = 2^(t - m) that meet the codes in fp16 (rounded to 11 bits)
// are at most 2^8 whatever the scales' sizes are, and the sum takes w / v_scale in fp32.
// bf16 caches: w is the sum of two bf16 (16 bits of it; the second product takes no time
// that HBM leaves).
#pragma once
#include <climits>
#include <cstdint>

#include "fa_cache_internal.h"
#include "sm103_ptx.cuh"

namespace {

using namespace fa_ptx;
using fa::CacheEntry;
using fa::CacheParams;

constexpr int kThreads = 32 * fa::kCacheWarps;
constexpr int kRows = fa::kCacheRows;
template <int D, int DV, bool Q8, bool FEW>
struct CacheCfg {
  static constexpr int CTAS = fa::cache_ctas(Q8, FEW);
  static constexpr int ES = Q8 ? 1 : 2;
  static constexpr int KC = fa::kCacheKeys;
  static constexpr int KROW = D * ES, VROW = DV * ES;  // bytes of a row
  static constexpr int KBYTES = KC * KROW, VBYTES = KC * VROW;
  static constexpr int SCALES = Q8 ? KC * 8 : 0;
  static constexpr int STAGE = KBYTES + VBYTES + SCALES;
  // For the join 8 rows of a warp's O lie in its stage that is free then, or else in a
  // buffer of their own.
  static constexpr int ROWS8 = 8 * DV * 4;
  static constexpr bool IN_STAGE = STAGE >= ROWS8;
  static constexpr int JOIN = IN_STAGE ? 0 : fa::kCacheWarps * ROWS8;
  static constexpr int ROOM = ((228 << 10) / CTAS - 1024 - 2560 - JOIN) / fa::kCacheWarps / STAGE;
  static constexpr int NS = ROOM > 6 ? 6 : ROOM;
  static constexpr int RING = NS * STAGE;  // per warp
  static constexpr int SMEM = fa::kCacheWarps * RING + JOIN;
  static_assert(NS >= 3 && STAGE % 16 == 0);
};

__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds4(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
// Four e4m3 codes -> four fp16, exactly.
__device__ __forceinline__ uint2 half4_of(uint32_t codes) {
  uint2 r;
  asm("{\n\t.reg .b16 c, u;\n\tmov.b32 {c, u}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(codes));
  return r;
}
template <bool Q8>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return Q8 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}
// Transposes 8 x 8 16-bit values: lane 4 r + i has (r, 2 i), (r, 2 i + 1) before, (2 i, r),
// (2 i + 1, r) after.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool Q8>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (Q8)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c * tanh(x / c) in log2 units of scores x without the softmax scale (see CapParams): by
// the polynomial where that serves all of the warp's, else by the form for any x.
template <int RT>
__device__ __forceinline__ void cap_scores(const fa::CapParams& c, float (&t)[RT][4]) {
  bool far = false;
  float y[RT][4];
#pragma unroll
  for (int u = 0; u < RT; ++u)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float v = t[u][x], s = v * v;
      far = far || s > c.small2;
      y[u][x] = v * (c.a[0] + s * (c.a[1] + s * (c.a[2] + s * (c.a[3] + s * c.a[4]))));
    }
  if (__any_sync(~0u, far)) {
#pragma unroll
    for (int u = 0; u < RT; ++u)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float v = t[u][x];
        if (!(v * v <= c.small2)) y[u][x] = c.log2c - 2.f * c.log2c * rcp(1.f + ex2(cap_top<true>(c.in * v)));
      }
  }
#pragma unroll
  for (int u = 0; u < RT; ++u)
#pragma unroll
    for (int x = 0; x < 4; ++x) t[u][x] = y[u][x];
}

struct __align__(16) Row {
  int at, last;  // position among the entry's keys (key j is at - j behind it), last key it may see
  int out;       // row of the result; -1: none; padding: -2 - row
  float slope;
};
// The softmax's reference follows a row's maximum when that has grown by more than this
// (log2 units: weights stay <= 256).
constexpr float kGrown = 8.f;

// FEW: the items have at most 8 rows, one tile of columns.  HIDES: some row of an item may not see
// a key that others see, or that lies in its chunk (several rows a sequence, or a window).
template <int D, int DV, bool Q8, bool FEW, bool HIDES>
__global__ void __launch_bounds__(kThreads, CacheCfg<D, DV, Q8, FEW>::CTAS) fa_cache_attn_kernel(const CacheParams p) {
  using C = CacheCfg<D, DV, Q8, FEW>;
  using Cursor = fa::CacheCursor<C::KC, kRows, fa::cache_item(FEW), HIDES>;
  constexpr int KC = C::KC, RT = FEW ? 1 : 2, MT = DV / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 s_ml[fa::kCacheWarps][kRows];
  __shared__ int s_free[fa::kCacheWarps];
  __shared__ Row s_row[fa::kCacheWarps][kRows];
  __shared__ Cursor s_load[fa::kCacheWarps];
  // Beside the prefixes' kernel (launched so that it may start with that): what comes before
  // both has completed; the end waits for that one, as the join waits for this one only.
  const auto share = fa::cache_share<KC, kRows, fa::cache_item(FEW), kThreads, HIDES>(p);
  if (share.begin >= share.end || share.start.at >= share.end) {
    if (blockIdx.x == 0) grid_previous();
    return;
  }

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int li = lane & 3, lr = lane >> 2;  // place in the quad, row (or column) of the quad
  const uint32_t ring = smem_u32(smem) + warp * C::RING;
  const int page_mask = (1 << p.page_log2) - 1, window = HIDES ? p.window : 0;

  // ------------------------------------------------------------ loads, ahead of the use
  // An item's chunks go round the warps, from another one on for each item of the share.
  Cursor& ld = s_load[warp];  // (in shared memory: registers are short)
  if (lane == 0) ld = share.start;
  __syncwarp();
  int lc = ld.c + warp, lc_end = ld.end(p, share.end), l_turn = 0;
  auto next_load = [&](int step) {  // to this warp's next chunk (lc >= lc_end: there is none)
    lc += step;
    while (lc >= lc_end) {
      __syncwarp();
      if (lane == 0) ld.next(p);
      __syncwarp();
      if (ld.at >= share.end) return;
      ++l_turn;
      lc = ld.c + ((warp - l_turn) & 3);
      lc_end = ld.end(p, share.end);
    }
  };
  auto page_of = [&]() {  // of the next chunk to load (its 16 keys lie in one)
    if (lc >= lc_end) return 0;
    const int col = ((ld.n.chunk0 + lc) * KC) >> p.page_log2;
    return __ldg(ld.e < p.S ? p.p_tables + (long long)ld.e * p.p_cols + col : p.tables + (long long)(ld.e - p.S) * p.cols + col);
  };
  next_load(0);
  int id = page_of();
  auto issue = [&](int stage) {
    if (lc < lc_end) {
      const uint32_t dst = ring + stage * C::STAGE;
      const int key = (ld.n.chunk0 + lc) * KC;
      const bool in_pool = (unsigned)id < (unsigned)p.pages;
      if (!in_pool) fa::cache_bad(p.status);
      const long long first = in_pool ? (((long long)id * p.Hkv + ld.h) << p.page_log2) | (key & page_mask) : 0;  // row in the pools
      // Rows [skip, rows) are loaded, the others are zero: those past the entry's end, and those before
      // the first key that any row sees, where a value may be anything.
      const int rows = in_pool ? ld.n.keys - key : 0, skip = HIDES ? ld.n.from - key : 0;
      constexpr int KP = C::KROW / 16, VP = C::VROW / 16;  // pieces of a row
      const int kr = lane / KP, kp = lane % KP, vr = lane / VP, vp = lane % VP;  // this lane's row and piece of the first copy
      const uint8_t* ks = p.K + (first + kr) * C::KROW + kp * 16;
      const uint8_t* vs = p.V + (first + vr) * C::VROW + vp * 16;
      const float* ss = nullptr;
      if constexpr (Q8) ss = (lane < 16 ? p.k_scale : p.v_scale) + first + (lane & 15);  // values' from lane 16 on
      const uint32_t kd = dst + kr * C::KROW + (KP >= 8 ? kp ^ ((kr & 1) << 2) : kp) * 16;
      auto vd = [&](int k) {
        const int row = vr + k * (32 / VP), sw = ((row >> 1) & 3) << 1;
        // (rows of 64 bytes: two to a line of 128, which is what the swizzle permutes)
        return dst + C::KBYTES + (VP >= 8 ? row * C::VROW + (vp ^ sw) * 16 : (row >> 1) * 128 + ((((row & 1) << 2) | vp) ^ sw) * 16);
      };
      if (rows >= KC && skip <= 0) {
#pragma unroll
        for (int k = 0; k < C::KBYTES / 512; ++k) cp16(kd + k * 512, ks + k * 512, true);
#pragma unroll
        for (int k = 0; k < C::VBYTES / 512; ++k) cp16(vd(k), vs + k * 512, true);
        if constexpr (Q8) cp4(dst + C::KBYTES + C::VBYTES + lane * 4, ss, true);
      } else {
#pragma unroll 1
        for (int k = 0; k < C::KBYTES / 512; ++k) {
          const int row = kr + k * (32 / KP);
          const bool ok = row >= skip && row < rows;
          cp16(kd + k * 512, ok ? ks + k * 512 : p.K, ok);
        }
#pragma unroll 1
        for (int k = 0; k < C::VBYTES / 512; ++k) {
          const int row = vr + k * (32 / VP);
          const bool ok = row >= skip && row < rows;
          cp16(vd(k), ok ? vs + k * 512 : p.V, ok);
        }
        if constexpr (Q8) {
          const bool ok = (lane & 15) >= skip && (lane & 15) < rows;
          cp4(dst + C::KBYTES + C::VBYTES + lane * 4, ok ? ss : p.k_scale, ok);
        }
      }
      next_load(fa::kCacheWarps);
      id = page_of();
    }
    cp_commit();
  };
#pragma unroll 1
  for (int s = 0; s < C::NS - 1; ++s) issue(s);
  int stage = 0, fill = C::NS - 1;

  // ------------------------------------------------------------ items
  Cursor it = share.start;
  int turn = 0;
  for (; it.at < share.end; it.next(p), ++turn) {
    const CacheEntry n = it.n;
    const bool is_prefix = it.e < p.S;
    const int c_end = it.end(p, share.end);

    // Q of rows lr and lr + 8 of the tile: the lane's pieces (16 channels in e4m3 calls, 8 in
    // bf16 ones)
    uint32_t q[RT][D / 8];
    float scale[RT];  // of those rows
#pragma unroll
    for (int u = 0; u < RT; ++u) {
      const fa::CacheRow r = fa::cache_row(p, n, it.r * kRows + lr + 8 * u);
      const uint16_t* src = p.Q + (((long long)r.b * p.Hq + it.h * p.G + r.g) * p.T + r.t) * D;
      constexpr int PIECE = Q8 ? 16 : 8;
#pragma unroll
      for (int k = 0; k < D / 8 / 4; ++k) {
        const int ch = (k * 8 / PIECE) * 4 * PIECE + li * PIECE + (k * 8) % PIECE;
        const uint4 v = r.valid ? __ldg(reinterpret_cast<const uint4*>(src + ch)) : make_uint4(0, 0, 0, 0);
        q[u][4 * k] = v.x, q[u][4 * k + 1] = v.y, q[u][4 * k + 2] = v.z, q[u][4 * k + 3] = v.w;
      }
      scale[u] = p.capped ? 1.f : p.scale_log2;
      if constexpr (Q8) {  // the row's largest value to [1, 2)
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) top = max(top, max(q[u][k] & 0x7fffu, (q[u][k] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        const int ex = min(max((int)(top >> 7), 1), 253);
        const float down = __uint_as_float((uint32_t)(254 - ex) << 23);
        scale[u] *= __uint_as_float((uint32_t)ex << 23);
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
          q[u][k] = pack_f16x2(__uint_as_float(q[u][k] << 16) * down, __uint_as_float(q[u][k] & 0xffff0000u) * down);
      }
    }
    // The rows whose scores this lane has: 2 li and 2 li + 1 of each tile of 8.  What is seldom
    // asked of a row lies in shared memory.
    __syncwarp();
    int all_from = INT_MIN;  // [all_from, all_to): keys that every row sees (but padding rows, whose part is none)
    if (lane < kRows) {
      const fa::CacheRow r = fa::cache_row(p, n, it.r * kRows + lane);
      const int pos = (is_prefix ? fa::cache_length(p, r.b) : n.keys) - p.T + r.t, out = (r.b * p.Hq + it.h * p.G + r.g) * p.T + r.t;
      Row& row = s_row[warp][lane];
      row.at = is_prefix ? n.keys + pos : pos;
      row.last = is_prefix ? n.keys - 1 : pos;
      row.out = !r.valid ? -1 : pos < 0 ? -2 - out : out;
      row.slope = p.slopes ? __ldg(p.slopes + it.h * p.G + r.g) * 1.4426950408889634f : 0.f;
      if (row.out >= 0) all_from = row.at - window + 1;
    }
    __syncwarp();
    all_from = window ? __reduce_max_sync(~0u, all_from) : 0;
    auto row_of = [&](int y) -> const Row& { return s_row[warp][2 * li + (y & 1) + 8 * (y >> 1)]; };
    float unit[2 * RT];
#pragma unroll
    for (int y = 0; y < 2 * RT; ++y) unit[y] = __shfl_sync(~0u, scale[y >> 1], (2 * li + (y & 1)) * 4);
    float m[2 * RT], l[2 * RT], o[RT][MT][4];
#pragma unroll
    for (int y = 0; y < 2 * RT; ++y) m[y] = -INFINITY, l[y] = 0.f;
#pragma unroll
    for (int u = 0; u < RT; ++u)
#pragma unroll
      for (int k = 0; k < MT; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[u][k][x] = 0.f;
    const int all_to = is_prefix ? n.keys : max(n.keys - p.T, 0) + 1;

    // The stages that held the last item's parts may be loaded again.
    if (turn) __syncthreads();
    for (int c = it.c + ((warp - turn) & 3); c < c_end; c += fa::kCacheWarps) {
      cp_wait<C::NS - 2>();
      __syncwarp();
      issue(fill);
      fill = fill + 1 == C::NS ? 0 : fill + 1;
      const uint32_t kb = ring + stage * C::STAGE, vb = kb + C::KBYTES, sb = vb + C::VBYTES;
      stage = stage + 1 == C::NS ? 0 : stage + 1;
      const int key0 = (n.chunk0 + c) * KC;

      // S^T: keys lr and lr + 8 of this lane, rows 2 li, 2 li + 1
      float t[RT][4];
#pragma unroll
      for (int u = 0; u < RT; ++u) t[u][0] = t[u][1] = t[u][2] = t[u][3] = 0.f;
#pragma unroll
      for (int k = 0; k < C::KROW / 64; ++k) {
        const int piece = 4 * k + li;
        const uint32_t at = kb + lr * C::KROW + (C::KROW >= 128 ? piece ^ ((lr & 1) << 2) : piece) * 16;
        const uint4 a = lds16(at), b = lds16(at + 8 * C::KROW);
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
        if constexpr (Q8) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int f = k * 8 + 2 * x;
            const uint2 ca = half4_of(wa[x]), cb = half4_of(wb[x]);
#pragma unroll
            for (int u = 0; u < RT; ++u) mma16<Q8>(t[u], ca.x, cb.x, ca.y, cb.y, q[u][f], q[u][f + 1]);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int f = k * 4 + 2 * x;
#pragma unroll
            for (int u = 0; u < RT; ++u) mma16<Q8>(t[u], wa[2 * x], wb[2 * x], wa[2 * x + 1], wb[2 * x + 1], q[u][f], q[u][f + 1]);
          }
        }
      }
      // scores in log2 units; element x: key lr + 8 (x >> 1), row 2 li + (x & 1)
      float ks[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f}, inv[2] = {1.f, 1.f};  // scale of the key, log2 of the value's, 1 / that
      if constexpr (Q8) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          ks[j] = lds4(sb + (lr + 8 * j) * 4);
          const float vs = lds4(sb + KC * 4 + (lr + 8 * j) * 4);
          // (a scale of 0, which no written row has, counts as 2^-69; a NaN reaches the
          // rows that see the key through t)
          const float a = lg2(fmaxf(vs, 0x1p-69f));
          inv[j] = ex2(-a);
          lv[j] = vs == vs ? a : vs;
        }
      }
#pragma unroll
      for (int u = 0; u < RT; ++u)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float v = t[u][x] * unit[2 * u + (x & 1)];
          if constexpr (Q8) v *= ks[x >> 1];
          t[u][x] = v;
        }
      if (p.capped) cap_scores(p.cap, t);
      if (p.slopes) {
#pragma unroll
        for (int y = 0; y < 2 * RT; ++y) {
          const Row row = row_of(y);
#pragma unroll
          for (int x = y & 1; x < 4; x += 2) t[y >> 1][x] -= row.slope * (float)(row.at - (key0 + lr + 8 * (x >> 1)));
        }
      }
      if constexpr (Q8) {  // before the mask: a hidden value's scale may be NaN
#pragma unroll
        for (int u = 0; u < RT; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x) t[u][x] += lv[x >> 1];
      }
      if (key0 + KC > all_to || key0 < all_from) {
#pragma unroll
        for (int y = 0; y < 2 * RT; ++y) {
          const Row row = row_of(y);
#pragma unroll
          for (int x = y & 1; x < 4; x += 2) {
            const int key = key0 + lr + 8 * (x >> 1);
            if (key > row.last || (window && row.at - key >= window)) t[y >> 1][x] = -INFINITY;
          }
        }
      }
      bool grown = false;
#pragma unroll
      for (int u = 0; u < RT; ++u)
#pragma unroll
        for (int x = 0; x < 4; ++x) grown = grown || t[u][x] > m[2 * u + (x & 1)] + kGrown;  // (-inf + 8: the first keys)
      if (__any_sync(~0u, grown)) {
#pragma unroll
        for (int y = 0; y < 2 * RT; ++y) {
          const int u = y >> 1, x = y & 1;
          float top = fmaxf(t[u][x], t[u][x + 2]);
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
          const float now = fmaxf(m[y], top), a = now == -INFINITY ? 1.f : ex2(m[y] - now);
          m[y] = now;
          l[y] *= a;
#pragma unroll
          for (int k = 0; k < MT; ++k) o[u][k][x] *= a, o[u][k][x + 2] *= a;
        }
      }
      uint32_t w[RT][2];  // P^T: keys 2 li, 2 li + 1 (+ 8) of row lr
      [[maybe_unused]] uint32_t rest[RT][2];  // (bf16) what their rounding left
#pragma unroll
      for (int u = 0; u < RT; ++u) {
        float e[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float ref = m[2 * u + (x & 1)];
          e[x] = ex2(t[u][x] - (ref == -INFINITY ? 0.f : ref));
          l[2 * u + (x & 1)] += Q8 ? e[x] * inv[x >> 1] : e[x];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t pair = pack2<Q8>(e[2 * j], e[2 * j + 1]);
          if constexpr (!Q8)
            rest[u][j] = turned(pack_bf16x2(e[2 * j] - __uint_as_float(pair << 16), e[2 * j + 1] - __uint_as_float(pair & 0xffff0000u)));
          w[u][j] = turned(pair);
        }
      }
      // bf16: a NaN or an infinity among the values of a chunk that some row does not see whole.  (In
      // e4m3 such a row's codes are 0, and its scale reaches those who see it through t.)
      [[maybe_unused]] bool careful = false;
      if constexpr (!Q8 && HIDES) {
        if (min(key0 + KC, n.keys) > all_to || key0 < all_from) {
          uint32_t bad = 0;
#pragma unroll
          for (int k = 0; k < C::VBYTES / 512; ++k) {
            const uint4 v = lds16(vb + k * 512 + lane * 16);
            bad |= not_finite2(v.x) | not_finite2(v.y) | not_finite2(v.z) | not_finite2(v.w);
          }
          careful = __any_sync(~0u, bad != 0);
        }
      }
      // O^T += V^T P^T: this lane's value rows 2 li, 2 li + 1, 8 + 2 li, 9 + 2 li
      auto mma_o = [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int u = 0; u < RT; ++u) {
          mma16<Q8>(o[u][k], a0, a1, a2, a3, w[u][0], w[u][1]);
          if constexpr (!Q8) mma16<Q8>(o[u][k], a0, a1, a2, a3, rest[u][0], rest[u][1]);
        }
      };
      // four channels of four rows
      auto four = [&](int k, uint32_t r0, uint32_t r1, uint32_t r8, uint32_t r9) {
        const uint2 a = half4_of(__byte_perm(r0, r1, 0x5140)), b = half4_of(__byte_perm(r8, r9, 0x5140));
        mma_o(k, a.x, a.y, b.x, b.y);
        const uint2 c = half4_of(__byte_perm(r0, r1, 0x7362)), d = half4_of(__byte_perm(r8, r9, 0x7362));
        mma_o(k + 1, c.x, c.y, d.x, d.y);
      };
      // The same with such values as 0, and NaN for the rows that see one of them in a channel.
      [[maybe_unused]] auto mma_seen = [&](int k, const uint32_t (&seen)[RT][2], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
        const uint32_t b0 = not_finite2(a0), b1 = not_finite2(a1), b2 = not_finite2(a2), b3 = not_finite2(a3), one = 0x3f803f80u;
        mma_o(k, a0 & ~b0, a1 & ~b1, a2 & ~b2, a3 & ~b3);
#pragma unroll
        for (int u = 0; u < RT; ++u) {
          float found[4] = {0.f, 0.f, 0.f, 0.f};
          mma16<Q8>(found, b0 & one, b1 & one, b2 & one, b3 & one, seen[u][0], seen[u][1]);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (found[x] > 0.f) o[u][k][x] = __uint_as_float(0x7fffffffu);
        }
      };
      if constexpr (Q8 && DV == 64) {  // 8 channels a lane: half a piece
        uint2 v[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int key = 2 * li + (y & 1) + (y >> 1) * 8;
          v[y] = lds8(vb + (key >> 1) * 128 + ((((key & 1) << 2) | (lr >> 1)) ^ (li << 1)) * 16 + (lr & 1) * 8);
        }
        four(0, v[0].x, v[1].x, v[2].x, v[3].x);
        four(2, v[0].y, v[1].y, v[2].y, v[3].y);
      } else {
        auto products = [&](auto mma) {
#pragma unroll
          for (int z = 0; z < C::VROW / 128; ++z) {
            uint4 v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int key = 2 * li + (y & 1) + (y >> 1) * 8;
              v[y] = lds16(vb + key * C::VROW + ((lr + 8 * z) ^ (li << 1)) * 16);
            }
            const uint32_t rows[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w}, {v[1].x, v[1].y, v[1].z, v[1].w},
                                      {v[2].x, v[2].y, v[2].z, v[2].w}, {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if constexpr (Q8)
                four(2 * x, rows[0][x], rows[1][x], rows[2][x], rows[3][x]);
              else
                mma(4 * z + x, __byte_perm(rows[0][x], rows[1][x], 0x5410), __byte_perm(rows[0][x], rows[1][x], 0x7632),
                    __byte_perm(rows[2][x], rows[3][x], 0x5410), __byte_perm(rows[2][x], rows[3][x], 0x7632));
            }
          }
        };
        if (!Q8 && HIDES && careful) {
          uint32_t seen[RT][2];  // as w: 1 where the row sees the key
#pragma unroll
          for (int u = 0; u < RT; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              seen[u][j] = turned((t[u][2 * j] == -INFINITY ? 0u : 0x3f80u) | (t[u][2 * j + 1] == -INFINITY ? 0u : 0x3f800000u));
          products([&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) { mma_seen(k, seen, a0, a1, a2, a3); });
        } else {
          products(mma_o);
        }
      }
    }

    // -------------------------------------------------------- the four warps' parts, added up
    // 8 rows of each lie in its stage that was read last and is loaded next, or in a buffer
    // of their own; each warp then adds up a quarter of the channels.
    auto rows8 = [&](int w) {
      return reinterpret_cast<float4*>(smem + (C::IN_STAGE ? w * C::RING + s_free[w] * C::STAGE : fa::kCacheWarps * C::RING + w * C::ROWS8)) + lane;
    };
    if (lane == 0) s_free[warp] = fill;
#pragma unroll
    for (int y = 0; y < 2 * RT; ++y) {
      l[y] += __shfl_xor_sync(~0u, l[y], 4);
      l[y] += __shfl_xor_sync(~0u, l[y], 8);
      l[y] += __shfl_xor_sync(~0u, l[y], 16);
      if (lr == 0) s_ml[warp][2 * li + (y & 1) + 8 * (y >> 1)] = make_float2(m[y], l[y]);
    }
    const bool whole = it.c == 0 && c_end == n.chunks && !p.joined;
    const long long slot = (long long)it.item + blockIdx.x;
#pragma unroll
    for (int u = 0; u < RT; ++u) {
      __syncthreads();
      float top[2], sum[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float2 v[fa::kCacheWarps];
        top[y] = -INFINITY;
#pragma unroll
        for (int w = 0; w < fa::kCacheWarps; ++w) {
          v[w] = s_ml[w][2 * li + y + 8 * u];
          top[y] = fmaxf(top[y], v[w].x);
        }
        sum[y] = 0.f;
#pragma unroll
        for (int w = 0; w < fa::kCacheWarps; ++w) sum[y] += v[w].y * (v[w].x == -INFINITY ? 1.f : ex2(v[w].x - top[y]));
        const float mine = m[2 * u + y], f = mine == -INFINITY ? 1.f : ex2(mine - top[y]);  // (without a finite m, O is 0 or NaN)
#pragma unroll
        for (int k = 0; k < MT; ++k) o[u][k][y] *= f, o[u][k][y + 2] *= f;
      }
      float4* dst = rows8(warp);
#pragma unroll
      for (int k = 0; k < MT; ++k) dst[k * 32] = make_float4(o[u][k][0], o[u][k][1], o[u][k][2], o[u][k][3]);
      __syncthreads();
      // this warp's share of the lane's channels: PER of them, from CH on in the row (their
      // order is that of the tiles' rows: see the products)
      constexpr int PER = DV / 32, RUN = Q8 || DV == 64 ? DV / 8 : 8;
      const int k0 = warp * PER, ch = (k0 / RUN) * 64 + lr * RUN + k0 % RUN;
      float c[2][PER] = {};
#pragma unroll
      for (int w = 0; w < fa::kCacheWarps; ++w) {
        const float4* src = rows8(w);
#pragma unroll
        for (int k = 0; k < PER; k += 2) {
          const float4 v = src[(k0 + k) / 2 * 32];
          c[0][k] += v.x, c[1][k] += v.y, c[0][k + 1] += v.z, c[1][k + 1] += v.w;
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int to = row_of(2 * u + y).out;
        if (to == -1) continue;
        const bool none = to < 0;  // a padding row: its part is none, whatever it scored a prefix's keys
        if (none) top[y] = -INFINITY, sum[y] = 0.f;
        const float g = none || (whole && sum[y] == 0.f) ? 0.f : whole ? 1.f / sum[y] : 1.f;
#pragma unroll
        for (int k = 0; k < PER; ++k) c[y][k] = g == 0.f ? 0.f : c[y][k] * g;
        if (whole) {
          const long long row = none ? -2 - to : to;
          if (lr == 0 && warp == 0) p.L[row] = sum[y] == 0.f ? -INFINITY : (top[y] + log2f(sum[y])) * 0.6931471805599453f;
          uint16_t* at = p.O + row * DV + ch;
          if constexpr (PER == 4)
            *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(c[y][0], c[y][1]), pack_bf16x2(c[y][2], c[y][3]));
          else
            *reinterpret_cast<uint32_t*>(at) = pack_bf16x2(c[y][0], c[y][1]);
        } else {
          const long long row = slot * kRows + 2 * li + y + 8 * u;
          if (lr == 0 && warp == 0) *reinterpret_cast<float2*>(p.parts.ml + row * 2) = make_float2(top[y], sum[y]);
          float* at = p.parts.part + row * DV + ch;
          if constexpr (PER == 4)
            *reinterpret_cast<float4*>(at) = make_float4(c[y][0], c[y][1], c[y][2], c[y][3]);
          else
            *reinterpret_cast<float2*>(at) = make_float2(c[y][0], c[y][1]);
        }
      }
    }
  }
  cp_wait<0>();
  grid_next();
  grid_previous();
}

template <int D, int DV, bool Q8, bool FEW, bool HIDES>
cudaError_t launch_rows(const CacheParams& p, int grid, cudaStream_t stream) {
  using C = CacheCfg<D, DV, Q8, FEW>;
  auto kernel = fa_cache_attn_kernel<D, DV, Q8, FEW, HIDES>;
  const cudaError_t e = fa::allow_dynamic_smem(reinterpret_cast<const void*>(kernel), C::SMEM);
  if (e != cudaSuccess) return e;
  // (Not so that it starts before the one before it ends, unless that is the prefixes': CTAs
  // that wait take the SMs of those that work; decoding 32 x 8192 in e4m3 95 -> 136 us.)
  if (p.sms) return fa::launch_next(kernel, dim3((unsigned)grid), kThreads, C::SMEM, stream, p);
  kernel<<<grid, kThreads, C::SMEM, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int DV, bool Q8>
cudaError_t launch_dims(const CacheParams& p, int grid, cudaStream_t stream) {
  // a prefix's items have the rows of several sequences
  const bool few = fa::cache_few(p.G * p.T, p.S > 0);
  // One row a sequence and no window: nothing is hidden but what lies past the ends.  (The code for
  // more costs such calls, in registers and in what is jumped over: 256 answers to 32768 tokens in bf16
  // took 172.5 us with it, 166.5 without; 16 to each of 8 prompts, heads of 64, 50.3 and 47.8.)
  if (p.T > 1 || p.window) return few ? launch_rows<D, DV, Q8, true, true>(p, grid, stream) : launch_rows<D, DV, Q8, false, true>(p, grid, stream);
  return few ? launch_rows<D, DV, Q8, true, false>(p, grid, stream) : launch_rows<D, DV, Q8, false, false>(p, grid, stream);
}

template <bool Q8>
cudaError_t launch_cache(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream) {
  if (d == 64) return dv == 64 ? launch_dims<64, 64, Q8>(p, grid, stream) : launch_dims<64, 128, Q8>(p, grid, stream);
  return dv == 64 ? launch_dims<128, 64, Q8>(p, grid, stream) : launch_dims<128, 128, Q8>(p, grid, stream);
}

}  // namespace
