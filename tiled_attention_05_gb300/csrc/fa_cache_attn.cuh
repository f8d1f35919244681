// Attention of the newest tokens over a paged key/value cache (fa_cache_attention).
//
//   O = softmax(scale q K^T, modified and masked) V,  L = logsumexp
// for a few rows per sequence.  Every key and value byte is read once and takes few
// operations, so HBM bounds it; the kernel's work is to keep enough loads in flight.
//
// Split.  The keys of all items (sequence or shared prefix, kv head, tile of 16 rows)
// form one list of chunks of 32 (e4m3) or 16 (bf16) keys, cut into equal shares, one
// for each CTA, whatever the lengths are.  A share that begins or ends inside an item
// leaves that item's part (unnormalised O, its reference and sum, in fp32) in the
// workspace, and a second kernel joins the parts in their order.  A prefix is an item
// list of its own, whose rows are those of all its sequences: its keys are read once
// per 16 rows, from HBM once.
//
// Warps.  Each of the CTA's four takes every fourth chunk of the share, through a ring
// of its own in shared memory (cp.async, no barrier between warps), and carries its own
// running maximum, sum and O.  The loads run ahead over the items' borders.  At an
// item's end the four are added up through shared memory.
//
// Products (mma.m16n8k16, fp32 accumulators; at 16 rows and these bytes they take a
// fraction of the time that HBM does).  S = Q K^T takes 8 keys as a tile's columns; the
// channels are dealt to the k slots so that a lane's share of a key is 16-byte pieces:
// lane i of a quad holds pieces i, i + 4, ...  The scores come out as the left operand
// of P V, whose columns are dealt so that a lane needs 16-byte pieces of a value row too.
// The pieces are swizzled in shared memory such that both reads are free of conflicts.
//
// e4m3 rows carry an fp32 scale.  Codes become fp16 exactly; q is brought to fp16 by its
// row's power of two (bf16's 8 bits fit into fp16's 11; what is 2^-24 of the row's
// largest value is lost).  The key's scale multiplies the score.  The value's goes into
// the exponent, t = score + log2(v_scale), and the softmax's reference is the maximum of
// t: the weights w = 2^(t - m) that meet the codes in fp16 (rounded to 11 bits) are at
// most 1 whatever the scales' sizes are, and the sum takes w / v_scale in fp32.
// bf16 caches: w is rounded to bf16, half a step being 2^-8 of a weight, as in the
// unmodified forward; the sum takes it unrounded.
#pragma once
#include <cstdint>

#include "fa_cache_internal.h"
#include "sm103_ptx.cuh"

namespace {

using namespace fa_ptx;
using fa::CacheEntry;
using fa::CacheParams;

constexpr int kThreads = 32 * fa::kCacheWarps;
constexpr int kRows = fa::kCacheRows;
// Shared memory for the rings of a CTA: two CTAs an SM, with 12 KB each for the join.
constexpr int kRingBytes = 100 << 10;

template <int D, int DV, bool Q8>
struct CacheCfg {
  static constexpr int ES = Q8 ? 1 : 2;
  static constexpr int KC = fa::cache_chunk_keys(Q8);
  static constexpr int KROW = D * ES, VROW = DV * ES;  // bytes of a row
  static constexpr int KBYTES = KC * KROW, VBYTES = KC * VROW;
  static constexpr int SCALES = Q8 ? KC * 8 : 0;
  static constexpr int STAGE = KBYTES + VBYTES + SCALES;
  static constexpr int FIT = kRingBytes / fa::kCacheWarps / STAGE;
  static constexpr int NS = FIT > 6 ? 6 : FIT;
  static constexpr int RING = NS * STAGE;  // per warp
  static constexpr int JOIN = (fa::kCacheWarps - 1) * 8 * DV * 4;  // 8 rows of three warps
  static constexpr int SMEM = fa::kCacheWarps * RING + JOIN;
  static_assert(NS >= 3 && STAGE % 16 == 0);
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  const uint2 v = lds8(a);
  return make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
}
// Two e4m3 codes (low 16 bits) -> two fp16, exactly.
__device__ __forceinline__ uint32_t half2_of(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 c, u;\n\tmov.b32 {c, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool Q8>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return Q8 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
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
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// c * tanh(x / c) in log2 units of a score x without the softmax scale (see CapParams).
__device__ __forceinline__ float capped(const fa::CapParams& c, float x) {
  const float u = x * x;
  if (u <= c.small2) return x * (c.a[0] + u * (c.a[1] + u * (c.a[2] + u * (c.a[3] + u * c.a[4]))));
  return c.log2c - 2.f * c.log2c * rcp(1.f + ex2(cap_top<true>(c.in * x)));
}

// FEW: the items have at most 8 rows (the upper half of the MMA's rows is not looked at).
template <int D, int DV, bool Q8, bool FEW>
__global__ void __launch_bounds__(kThreads, fa::kCacheCtasPerSm) fa_cache_attn_kernel(const CacheParams p) {
  using C = CacheCfg<D, DV, Q8>;
  using Cursor = fa::CacheCursor<C::KC, kRows>;
  constexpr int KC = C::KC, NT = KC / 8, HALVES = FEW ? 1 : 2, ON = DV / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 s_ml[2][fa::kCacheWarps][kRows];
  grid_next();
  grid_previous();
  const bool groups_ok = fa::cache_groups_ok(p);
  const auto share = fa::cache_share<KC, kRows, kThreads>(p, groups_ok);
  if (share.begin >= share.end) return;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int li = lane & 3, lr = lane >> 2;  // place in the quad, row (or column) of the quad
  const uint32_t ring = smem_u32(smem) + warp * C::RING;
  float4* join = reinterpret_cast<float4*>(smem + fa::kCacheWarps * C::RING);
  const int page_mask = (1 << p.page_log2) - 1;

  // ------------------------------------------------------------ loads, ahead of the use
  Cursor ld = share.start;
  int id0 = 0, id1 = 0;
  // the pages of the next chunk to load: its keys lie in one page, or in two by halves of 16
  auto fetch_ids = [&]() {
    if (ld.at >= share.end) return;
    const int key = (ld.n.chunk0 + ld.c) * KC;
    const int* tab = ld.e < p.S ? p.p_tables + (long long)ld.e * p.p_cols : p.tables + (long long)(ld.e - p.S) * p.cols;
    const int cols = ld.e < p.S ? p.p_cols : p.cols;
    const int c0 = key >> p.page_log2, c1 = min((key + 16) >> p.page_log2, cols - 1);
    id0 = __ldg(tab + c0);
    id1 = KC > 16 ? __ldg(tab + c1) : id0;
  };
  auto issue = [&](int stage) {
    if (ld.at < share.end) {
      const uint32_t dst = ring + stage * C::STAGE;
      const int key = (ld.n.chunk0 + ld.c) * KC, left = ld.n.keys - key;
      const bool ok0 = (unsigned)id0 < (unsigned)p.pages, ok1 = (unsigned)id1 < (unsigned)p.pages;
      if (!ok0 || (!ok1 && left > 16)) fa::cache_bad(p.status);
      // first rows of the two halves in the pools
      const long long r0 = ok0 ? ((((long long)id0 * p.Hkv + ld.h) << p.page_log2) | (key & page_mask)) : 0;
      const long long r1 = ok1 ? ((((long long)id1 * p.Hkv + ld.h) << p.page_log2) | ((key + 16) & page_mask)) : 0;
      const int n0 = ok0 ? min(left, 16) : 0, n1 = KC > 16 && ok1 ? left - 16 : 0;  // rows to load of each
      constexpr int KP = C::KROW / 16, VP = C::VROW / 16;  // pieces of a row
#pragma unroll
      for (int k = 0; k < C::KBYTES / 512; ++k) {
        const int row = (k * 32 + lane) / KP, piece = lane % KP, in = row & 15;
        const bool up = KC > 16 && (k * 32) / KP >= 16, ok = in < (up ? n1 : n0);
        const uint8_t* src = p.K + ((up ? r1 : r0) + in) * C::KROW + piece * 16;
        cp16(dst + row * C::KROW + (KP >= 8 ? piece ^ ((row & 1) << 2) : piece) * 16, ok ? src : p.K, ok);
      }
#pragma unroll
      for (int k = 0; k < C::VBYTES / 512; ++k) {
        const int row = (k * 32 + lane) / VP, piece = lane % VP, in = row & 15;
        const bool up = KC > 16 && (k * 32) / VP >= 16, ok = in < (up ? n1 : n0);
        const uint8_t* src = p.V + ((up ? r1 : r0) + in) * C::VROW + piece * 16;
        // (rows of 64 bytes: two to a line of 128, which is what the swizzle permutes)
        const uint32_t at = VP >= 8 ? row * C::VROW + (piece ^ (((row >> 1) & 3) << 1)) * 16
                                    : (row >> 1) * 128 + ((((row & 1) << 2) | piece) ^ (((row >> 1) & 3) << 1)) * 16;
        cp16(dst + C::KBYTES + at, ok ? src : p.V, ok);
      }
      if constexpr (Q8) {
        const int in = lane & 15;
        const bool up = lane >= 16, ok = in < (up ? n1 : n0);
        const long long at = ok ? (up ? r1 : r0) + in : 0;
        cp4(dst + C::KBYTES + C::VBYTES + lane * 4, p.k_scale + at, ok);
        cp4(dst + C::KBYTES + C::VBYTES + KC * 4 + lane * 4, p.v_scale + at, ok);
      }
      ld.advance(p, groups_ok, fa::kCacheWarps);
      fetch_ids();
    }
    cp_commit();
  };
  if (warp) ld.advance(p, groups_ok, warp);
  fetch_ids();
#pragma unroll
  for (int s = 0; s < C::NS - 1; ++s) issue(s);
  int stage = 0, fill = C::NS - 1;

  // ------------------------------------------------------------ items
  Cursor it = share.start;
  int item = share.item, turn = 0;
  long long mine = share.begin + warp;  // this warp's next chunk
  while (it.at < share.end) {
    const CacheEntry n = it.n;
    const bool is_prefix = it.e < p.S;
    const long long left_in_share = share.end - it.at;
    const int c_end = left_in_share < n.chunks - it.c ? it.c + (int)left_in_share : n.chunks;
    const long long seg_end = it.at + (c_end - it.c);

    // the rows of this lane: lr and lr + 8 of the tile
    int abs0[HALVES];      // row's position among the entry's keys: key j is `abs - j` behind it
    int last[HALVES];      // last key it may see
    float slope[HALVES], unit[HALVES];
    uint32_t q[HALVES][D / 8];
#pragma unroll
    for (int u = 0; u < HALVES; ++u) {
      const fa::CacheRow r = fa::cache_row(p, n, it.r * kRows + lr + 8 * u);
      const int pos = fa::cache_length(p, r.b) - p.T + r.t;
      abs0[u] = is_prefix ? n.keys + pos : pos;
      last[u] = is_prefix ? n.keys - 1 : pos;
      const int head = it.h * p.G + r.g;
      slope[u] = p.slopes ? __ldg(p.slopes + head) * 1.4426950408889634f : 0.f;
      const uint16_t* src = p.Q + (((long long)r.b * p.Hq + head) * p.T + r.t) * D;
      uint32_t w[D / 8];
      // the channels of this lane: pieces of 16 (e4m3) or 8 (bf16)
      constexpr int PIECE = Q8 ? 16 : 8;
#pragma unroll
      for (int k = 0; k < D / 8 / 4; ++k) {
        const int ch = (k * 8 / PIECE) * 4 * PIECE + li * PIECE + (k * 8) % PIECE;
        const uint4 v = r.valid ? __ldg(reinterpret_cast<const uint4*>(src + ch)) : make_uint4(0, 0, 0, 0);
        w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
      }
      unit[u] = p.capped ? 1.f : p.scale_log2;
      if constexpr (Q8) {  // the row's largest value to [1, 2)
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        const int ex = min(max((int)(top >> 7), 1), 253);
        const float down = __uint_as_float((uint32_t)(254 - ex) << 23);
        unit[u] *= __uint_as_float((uint32_t)ex << 23);
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
          w[k] = pack_f16x2(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xffff0000u) * down);
      }
#pragma unroll
      for (int k = 0; k < D / 8; ++k) q[u][k] = w[k];
    }
    float m[HALVES], l[HALVES], o[ON][2 * HALVES];
#pragma unroll
    for (int u = 0; u < HALVES; ++u) m[u] = -INFINITY, l[u] = 0.f;
#pragma unroll
    for (int k = 0; k < ON; ++k)
#pragma unroll
      for (int x = 0; x < 2 * HALVES; ++x) o[k][x] = 0.f;
    // keys that every row of the item sees, without a window: [0, seen_by_all)
    const int seen_by_all = is_prefix ? n.keys : max(n.keys - p.T, 0) + 1;

    for (; mine < seg_end; mine += fa::kCacheWarps) {
      cp_wait<C::NS - 2>();
      __syncwarp();
      issue(fill);
      fill = fill + 1 == C::NS ? 0 : fill + 1;
      const uint32_t kb = ring + stage * C::STAGE, vb = kb + C::KBYTES, sb = vb + C::VBYTES;
      stage = stage + 1 == C::NS ? 0 : stage + 1;
      const int key0 = (n.chunk0 + it.c + (int)(mine - it.at)) * KC;

      float t[NT][2 * HALVES];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const int key = j * 8 + lr;
#pragma unroll
        for (int k = 0; k < C::KROW / 64; ++k) {
          const int piece = 4 * k + li;
          const uint4 v = lds16(kb + key * C::KROW + (C::KROW >= 128 ? piece ^ ((lr & 1) << 2) : piece) * 16);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          if constexpr (Q8) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int f = k * 8 + 2 * x;
              mma16<Q8>(s, q[0][f], FEW ? 0u : q[HALVES - 1][f], q[0][f + 1], FEW ? 0u : q[HALVES - 1][f + 1],
                        half2_of(w[x]), half2_of(w[x] >> 16));
            }
          } else {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int f = k * 4 + 2 * x;
              mma16<Q8>(s, q[0][f], FEW ? 0u : q[HALVES - 1][f], q[0][f + 1], FEW ? 0u : q[HALVES - 1][f + 1],
                        w[2 * x], w[2 * x + 1]);
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 2 * HALVES; ++x) t[j][x] = s[x];
      }
      // scores in log2 units
      float inv[NT][2];  // 1 / v_scale
      float lv[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float2 ks = make_float2(1.f, 1.f);
        if constexpr (Q8) {
          ks = lds_f2(sb + (j * 8 + 2 * li) * 4);
          const float2 vs = lds_f2(sb + KC * 4 + (j * 8 + 2 * li) * 4);
          // (a scale of 0, which no written row has, counts as 2^-69; a NaN reaches the
          // rows that see the key through t)
          const float a = lg2(fmaxf(vs.x, 0x1p-69f)), b = lg2(fmaxf(vs.y, 0x1p-69f));
          inv[j][0] = ex2(-a), inv[j][1] = ex2(-b);
          lv[j][0] = vs.x == vs.x ? a : vs.x, lv[j][1] = vs.y == vs.y ? b : vs.y;
        }
#pragma unroll
        for (int x = 0; x < 2 * HALVES; ++x) {
          const int u = x >> 1;
          float v = t[j][x] * unit[u];
          if constexpr (Q8) v *= (x & 1) ? ks.y : ks.x;
          if (p.capped) v = capped(p.cap, v);
          t[j][x] = v;
        }
      }
      if (p.slopes) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int x = 0; x < 2 * HALVES; ++x)
            t[j][x] -= slope[x >> 1] * (float)(abs0[x >> 1] - (key0 + j * 8 + 2 * li + (x & 1)));
      }
      if (p.window || key0 + KC > seen_by_all) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int x = 0; x < 2 * HALVES; ++x) {
            const int key = key0 + j * 8 + 2 * li + (x & 1), u = x >> 1;
            if (key > last[u] || (p.window && abs0[u] - key >= p.window)) t[j][x] = -INFINITY;
          }
      }
      float a[HALVES];
      bool grew = false;
#pragma unroll
      for (int u = 0; u < HALVES; ++u) {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if constexpr (Q8) {
            t[j][2 * u] += lv[j][0];
            t[j][2 * u + 1] += lv[j][1];
          }
          top = fmaxf(top, fmaxf(t[j][2 * u], t[j][2 * u + 1]));
        }
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const float now = fmaxf(m[u], top);
        a[u] = now == -INFINITY ? 1.f : ex2(m[u] - now);
        grew = grew || now > m[u];
        m[u] = now;
      }
      if (__any_sync(~0u, grew)) {
#pragma unroll
        for (int u = 0; u < HALVES; ++u) {
          l[u] *= a[u];
#pragma unroll
          for (int k = 0; k < ON; ++k) o[k][2 * u] *= a[u], o[k][2 * u + 1] *= a[u];
        }
      }
#pragma unroll
      for (int u = 0; u < HALVES; ++u) {
        const float base = m[u] == -INFINITY ? 0.f : m[u];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float w0 = ex2(t[j][2 * u] - base), w1 = ex2(t[j][2 * u + 1] - base);
          l[u] += Q8 ? w0 * inv[j][0] + w1 * inv[j][1] : w0 + w1;
          t[j][2 * u] = w0, t[j][2 * u + 1] = w1;
        }
      }
      // O += P V, 16 keys a step: this lane's value rows 2 li, 2 li + 1, 8 + 2 li, 9 + 2 li
#pragma unroll
      for (int j = 0; j < NT; j += 2) {
        const uint32_t p0 = pack2<Q8>(t[j][0], t[j][1]), p2 = pack2<Q8>(t[j + 1][0], t[j + 1][1]);
        uint32_t p1 = 0, p3 = 0;
        if constexpr (!FEW) {
          p1 = pack2<Q8>(t[j][HALVES], t[j][HALVES + 1]);
          p3 = pack2<Q8>(t[j + 1][HALVES], t[j + 1][HALVES + 1]);
        }
        auto mma_o = [&](int k, uint32_t b0, uint32_t b1) {
          float c[4] = {o[k][0], o[k][1], FEW ? 0.f : o[k][2 * HALVES - 2], FEW ? 0.f : o[k][2 * HALVES - 1]};
          mma16<Q8>(c, p0, p1, p2, p3, b0, b1);
          o[k][0] = c[0], o[k][1] = c[1];
          if constexpr (!FEW) o[k][2] = c[2], o[k][3] = c[3];
        };
        if constexpr (Q8 && DV == 64) {
          // 8 channels a lane: half a piece
          uint2 v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int key = j * 8 + 2 * li + (y & 1) + (y >> 1) * 8;
            v[y] = lds8(vb + (key >> 1) * 128 + ((((key & 1) << 2) | (lr >> 1)) ^ (li << 1)) * 16 + (lr & 1) * 8);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a0 = x ? v[0].y : v[0].x, a1 = x ? v[1].y : v[1].x, a2 = x ? v[2].y : v[2].x,
                           a3 = x ? v[3].y : v[3].x;
            const uint32_t lo0 = __byte_perm(a0, a1, 0x5140), hi0 = __byte_perm(a0, a1, 0x7362);
            const uint32_t lo1 = __byte_perm(a2, a3, 0x5140), hi1 = __byte_perm(a2, a3, 0x7362);
            mma_o(4 * x, half2_of(lo0), half2_of(lo1));
            mma_o(4 * x + 1, half2_of(lo0 >> 16), half2_of(lo1 >> 16));
            mma_o(4 * x + 2, half2_of(hi0), half2_of(hi1));
            mma_o(4 * x + 3, half2_of(hi0 >> 16), half2_of(hi1 >> 16));
          }
        } else {
#pragma unroll
          for (int z = 0; z < C::VROW / 128; ++z) {
            uint4 v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int key = j * 8 + 2 * li + (y & 1) + (y >> 1) * 8;
              v[y] = lds16(vb + key * C::VROW + ((lr + 8 * z) ^ (li << 1)) * 16);
            }
            const uint32_t w[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w}, {v[1].x, v[1].y, v[1].z, v[1].w},
                                      {v[2].x, v[2].y, v[2].z, v[2].w}, {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if constexpr (Q8) {
                const uint32_t lo0 = __byte_perm(w[0][x], w[1][x], 0x5140), hi0 = __byte_perm(w[0][x], w[1][x], 0x7362);
                const uint32_t lo1 = __byte_perm(w[2][x], w[3][x], 0x5140), hi1 = __byte_perm(w[2][x], w[3][x], 0x7362);
                mma_o(4 * x, half2_of(lo0), half2_of(lo1));
                mma_o(4 * x + 1, half2_of(lo0 >> 16), half2_of(lo1 >> 16));
                mma_o(4 * x + 2, half2_of(hi0), half2_of(hi1));
                mma_o(4 * x + 3, half2_of(hi0 >> 16), half2_of(hi1 >> 16));
              } else {
                mma_o(8 * z + 2 * x, __byte_perm(w[0][x], w[1][x], 0x5410), __byte_perm(w[2][x], w[3][x], 0x5410));
                mma_o(8 * z + 2 * x + 1, __byte_perm(w[0][x], w[1][x], 0x7632), __byte_perm(w[2][x], w[3][x], 0x7632));
              }
            }
          }
        }
      }
    }

    // -------------------------------------------------------- the four warps' parts, added up
    // One warp, another one for each item, adds the other three's to its own; these go on
    // to the next item meanwhile (at most to its end: s_ml has two sides, and the buffer
    // is written only behind a barrier that the adding warp has reached).
    const int adder = turn & 3, side = turn & 1;
    ++turn;
#pragma unroll
    for (int u = 0; u < HALVES; ++u) {
      l[u] += __shfl_xor_sync(~0u, l[u], 1);
      l[u] += __shfl_xor_sync(~0u, l[u], 2);
      if (li == 0) s_ml[side][warp][lr + 8 * u] = make_float2(m[u], l[u]);
    }
    const bool whole = it.c == 0 && c_end == n.chunks && !p.joined;
    const long long slot = (long long)item + blockIdx.x;
#pragma unroll
    for (int u = 0; u < HALVES; ++u) {
      __syncthreads();
      const int row = lr + 8 * u;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < fa::kCacheWarps; ++w) top = fmaxf(top, s_ml[side][w][row].x);
      const float f = m[u] == -INFINITY ? 1.f : ex2(m[u] - top);  // (without a finite m, O is 0 or NaN)
#pragma unroll
      for (int k = 0; k < ON; ++k) o[k][2 * u] *= f, o[k][2 * u + 1] *= f;
      if (warp != adder) {
        float4* dst = join + ((warp - adder - 1) & 3) * (ON * 16) + lane;
#pragma unroll
        for (int k = 0; k < ON; k += 2)
          dst[k * 16] = make_float4(o[k][2 * u], o[k][2 * u + 1], o[k + 1][2 * u], o[k + 1][2 * u + 1]);
      }
      __syncthreads();
      if (warp == adder) {
#pragma unroll
        for (int w = 0; w < fa::kCacheWarps - 1; ++w)
#pragma unroll
          for (int k = 0; k < ON; k += 2) {
            const float4 v = join[w * (ON * 16) + lane + k * 16];
            o[k][2 * u] += v.x, o[k][2 * u + 1] += v.y, o[k + 1][2 * u] += v.z, o[k + 1][2 * u + 1] += v.w;
          }
#pragma unroll
        for (int w = 0; w < fa::kCacheWarps; ++w) {
          const float2 v = s_ml[side][w][row];
          sum += v.y * (v.x == -INFINITY ? 1.f : ex2(v.x - top));
        }
        const int at = it.r * kRows + row;
        if (at < n.rows) {
          const fa::CacheRow r = fa::cache_row(p, n, at);
          if (fa::cache_length(p, r.b) - p.T + r.t < 0) {  // a padding row
            sum = 0.f;
#pragma unroll
            for (int k = 0; k < ON; ++k) o[k][2 * u] = o[k][2 * u + 1] = 0.f;
          }
          // the lane's channels: those of columns 2 li and 2 li + 1 of the output tiles
          constexpr int RUN = Q8 || DV == 64 ? DV / 8 : 8;
          if (whole) {
            const long long out = ((long long)r.b * p.Hq + it.h * p.G + r.g) * p.T + r.t;
            const float g = sum == 0.f ? 0.f : 1.f / sum;
            if (li == 0) p.L[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int k = 0; k < ON; k += 8) {
                uint32_t w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) w[x] = pack_bf16x2(o[k + 2 * x][2 * u + y] * g, o[k + 2 * x + 1][2 * u + y] * g);
                *reinterpret_cast<uint4*>(p.O + out * DV + (k / RUN) * 64 + (2 * li + y) * RUN + k % RUN) =
                    make_uint4(w[0], w[1], w[2], w[3]);
              }
          } else {
            if (li == 0) *reinterpret_cast<float2*>(p.parts.ml + (slot * kRows + row) * 2) = make_float2(top, sum);
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int k = 0; k < ON; k += 4)
                *reinterpret_cast<float4*>(p.parts.part + (slot * kRows + row) * DV + (k / RUN) * 64 + (2 * li + y) * RUN + k % RUN) =
                    make_float4(o[k][2 * u + y], o[k + 1][2 * u + y], o[k + 2][2 * u + y], o[k + 3][2 * u + y]);
          }
        }
      }
    }
    item += c_end == n.chunks;
    const int old = it.e;
    it.advance(p, groups_ok, c_end - it.c);
    // (entries without work have items of their own number too)
    for (int e = old + 1; e < it.e && e < p.entries; ++e) item += p.Hkv * fa::cache_entry<KC>(p, e, groups_ok).tiles(kRows);
  }
  cp_wait<0>();
}

template <int D, int DV, bool Q8>
cudaError_t launch_dims(const CacheParams& p, int grid, cudaStream_t stream) {
  using C = CacheCfg<D, DV, Q8>;
  // a prefix's items have the rows of several sequences
  auto kernel = p.S == 0 && p.G * p.T <= 8 ? fa_cache_attn_kernel<D, DV, Q8, true> : fa_cache_attn_kernel<D, DV, Q8, false>;
  const cudaError_t e = fa::allow_dynamic_smem(reinterpret_cast<const void*>(kernel), C::SMEM);
  if (e != cudaSuccess) return e;
  return fa::launch_next(kernel, dim3((unsigned)grid), kThreads, C::SMEM, stream, p);
}

template <bool Q8>
cudaError_t launch_cache(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream) {
  if (d == 64) return dv == 64 ? launch_dims<64, 64, Q8>(p, grid, stream) : launch_dims<64, 128, Q8>(p, grid, stream);
  return dv == 64 ? launch_dims<128, 64, Q8>(p, grid, stream) : launch_dims<128, 128, Q8>(p, grid, stream);
}

}  // namespace
