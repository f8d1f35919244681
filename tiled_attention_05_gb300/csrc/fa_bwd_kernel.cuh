// Backward main kernel of tiled exact attention on sm_103a (the plain instances
// and the other two kernels are in fa_bwd.cu, the score-modified instances in
// fa_scored_bwd_*.cu).
//
// Method ("What Ordinary Autograd Saves", section "Why this is
// FlashAttention's second idea"; "Backward Pass Implementation", section "The
// Recomputation Strategy"): only O and the row statistic L survive the
// forward; every score/probability tile is rebuilt on chip from Q, K and L.
// With D_i = rowsum(dO_i * O_i):
//     P = exp(scale * Q K^T - L),  dP = dO V^T,  dS = P * (dP - D),
//     dV += P^T dO,  dK += dS^T Q * scale,  dQ += dS K * scale.
//
// Three kernels:
//   fa_bwd_pre   D = rowsum(dO * O), L in log2 units (+inf on padding rows so
//                that their probabilities vanish), zero the fp32 dQ
//                accumulator and the split items' counters.  HBM-bound, a row
//                per group of dv / 8 lanes.
//   fa_bwd_main  one CTA per (batch, kv head, 128-key tile) -- without a causal
//                mask, a short last round of tiles runs as two CTAs per tile,
//                each over half of its query tiles, whose fp32 dK / dV meet in
//                the workspace -- K and V stay in
//                shared memory; the CTA walks the G query heads of its group
//                and the 128-row query tiles that can see its keys (causal:
//                from the diagonal on; with a sliding window of W keys, up to
//                the last row whose window still reaches the tile), keeping dK
//                and dV in TMEM for the whole walk and adding each tile's dQ
//                into the fp32 accumulator in global memory.
//   fa_dq_cast   dQ = bf16(scale * accumulator).  HBM-bound.
//
// fa_bwd_main roles (512 threads, four warpgroups):
//   warp 0      TMA: K, V once; then Q_t (+ the tile's L and D slices by 1-D
//               bulk copy) through a 2-deep ring and dO_t through one buffer
//               (3-deep and 2 buffers at d = dv = 64).
//   warp 1      tcgen05 issuer, per tile t:
//                 dP^T = V dO_t^T       -> TMEM [128,256)
//                 dV  += P^T dO_t       A = P^T from TMEM (bf16, written over S^T)
//                 S^T(t+1) = K Q_{t+1}^T -> TMEM [0,128)     (key rows = lanes)
//                 dK  += dS^T Q_t       A = dS^T from TMEM (bf16, written over dP^T)
//                 dQ_t = dS K           -> TMEM [128,128+d), or at d = 64 the free
//                                        columns after dK; A = the dS bytes in
//                                        shared memory read MN-major; B = K read MN-major
//               relying on in-order MMA execution, not on waits, wherever a
//               later MMA overwrites columns an earlier one reads.  At
//               d = dv = 64 it checks only P and dS per tile: one elementwise
//               thread and the dQ warps vouch for Q_{t+1}, dO_{t+1} and the
//               drained dQ columns.
//   warps 4..11 two elementwise warpgroups (thread = key row = TMEM lane; group
//               w owns query columns [64w, 64w+64)): P = exp2(S*scale*log2e - L2)
//               with masks -> TMEM; dS = P * (dP - D) -> shared memory (for the
//               dQ MMA) and, packed, into TMEM over dP^T (for the dK MMA).
//               Epilogue: dV and dK*scale -> bf16 -> TMA store.
//   warps 12..15 dQ warpgroup (thread = query row): each warp copies its 32
//               rows of dQ_t out of TMEM into registers, releases the columns,
//               then stages two 32-column chunks at a time in its own
//               128B-swizzled fp32 slots and adds each chunk into the fp32
//               accumulator in global memory with one TMA bulk reduce-add
//               (32 x 32 box); no cross-warp synchronisation.  At d = 128 it
//               takes registers from the producer / MMA warpgroup (setmaxnreg)
//               to hold a whole dQ row.
// TMEM columns: S^T/P^T [0,128), dP^T/dS^T/dQ [128,256), dV [256,256+dv), dK [256+dv, 256+dv+d);
// at d = 64 dQ moves to [256+dv+d, 256+dv+2d).
//
// Score-modified instances (SCORE >= 0) rebuild the modified scores as the
// forward does (fa_fwd_kernel.cuh).  The cap's derivative is 1 - tanh^2 =
// 4 e r^2 with the e = exp(2 s / c) and r = 1 / (1 + e) already at hand (with the
// polynomial 1 - (x / c)^2), so the fp32 P kept for dS is P times a quarter of it
// and the factor 4 joins the scale of dK and dQ: no further registers.  The
// distance bias has no gradient (its slopes are constants).  Masks: query rows
// [from, to] see this thread's key, from the mask plan or from the two lines of
// causal mask and window; a plan whose intervals are not in order is looked up
// row by row instead.  Where there are few key tiles of unequal work, the
// heaviest run in parts (fa::scored_split).  Bounded as the plain form is, with
// a longer elementwise phase: 32 / 8 heads of 128, T 8192, causal, 970 us plain,
// 977 with slopes, 1152 with a cap, 1228 with both.
#pragma once
#include <cstdint>
#include <type_traits>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

using namespace fa_ptx;

namespace {

constexpr int BM = fa::kTile;  // query rows per tile
constexpr int BN = fa::kTile;  // keys per CTA
constexpr int kThreads = 512;
// Register split of fa_bwd_main at d = 128 (see the kernel): every thread
// starts with kRegsLaunch; the producer / MMA warpgroup drops to kRegsLow and
// the dQ warpgroup rises to kRegsHigh, the two elementwise warpgroups keep
// kRegsLaunch.
constexpr int kRegsLaunch = 65536 / kThreads;  // 128
constexpr int kRegsLow = 80;
constexpr int kRegsHigh = 2 * kRegsLaunch - kRegsLow;  // 176
template <int HD>
constexpr bool kSplitRegs = HD == 128;
static_assert(kRegsLow % 8 == 0 && kRegsHigh % 8 == 0 && kRegsHigh <= 256, "setmaxnreg operands");

// HD: head size of Q and K; HDV: head size of V, O and dO.
template <int HD, int HDV>
struct BwdCfg {
  // d = dv = 64 leaves shared memory for deeper Q and dO rings.  Loads then
  // land a tile earlier, and other roles can vouch for three of the MMA
  // thread's five checks per tile (see the kernel): one elementwise thread
  // checks Q(t+1) before it releases P(t) and dO(t+1) before it releases
  // dS(t), and the dQ warps arrive on ds_ready(t+1) once dQ(t) is drained.
  static constexpr bool VOUCH = HD == 64 && HDV == 64;
  static constexpr int NQ = VOUCH ? 3 : 2;   // Q tiles (with their L and D slices) in flight
  static constexpr int NDO = VOUCH ? 2 : 1;  // dO tiles in flight
  static constexpr int QK_TILE = 128 * HD * 2;   // one Q or K tile (bf16)
  static constexpr int VO_TILE = 128 * HDV * 2;  // one V or dO tile (bf16)
  static constexpr int DS_BYTES = BN * BM * 2;
  static constexpr int STG_SLOT = 32 * 32 * 4;  // one warp's 32 rows x 32 fp32 columns
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + QK_TILE;
  static constexpr int OFF_Q = OFF_V + VO_TILE;         // [NQ]
  static constexpr int OFF_DO = OFF_Q + NQ * QK_TILE;   // [NDO]
  static constexpr int OFF_DS = OFF_DO + NDO * VO_TILE;
  // Epilogue staging of dV and dK over the Q ring and the dO buffer (idle by then).
  static constexpr int OFF_DV_STAGE = OFF_Q;
  static constexpr int OFF_DK_STAGE = OFF_Q + (QK_TILE > VO_TILE ? QK_TILE : VO_TILE);
  static_assert(OFF_DK_STAGE + QK_TILE <= OFF_DS, "dV / dK staging fits in the Q ring and dO buffer");
  static constexpr int OFF_STG = OFF_DS + DS_BYTES;       // [4 warps][2] dQ staging slots
  static constexpr int OFF_LSE = OFF_STG + 8 * STG_SLOT;  // [NQ][128] fp32
  static constexpr int OFF_DELTA = OFF_LSE + NQ * 512;   // [NQ][128] fp32
  static constexpr int OFF_BAR = OFF_DELTA + NQ * 512;
  static constexpr int NBAR = 24;
  static_assert(1 + 2 * NQ + 2 * NDO + 8 <= NBAR, "barrier slots");
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
  static_assert(SMEM <= 232448, "shared memory budget");
};

// Epilogue of one fp32 accumulator of W columns in TMEM (dV or dK): this
// thread's key row r, the warpgroup's half of the columns (wg), times `mul`,
// as bf16 into a 128-row, 128B-swizzled staging tile for the TMA store.
// `have` is false when the CTA saw no query tile: the rows are zero.
// `add` (optional): the same row's partial sums from the other half of a
// split item, this warpgroup's columns, added before the scaling; or, with `all`, those
// of all n_add parts (its own among them), add_stride floats apart, added in their
// order, whichever of them is the last to finish, so that the sum is the same every time.
// The loops stay rolled: what this code takes up moves the main loop's (cap and slopes,
// T 8192, 32 / 8 heads of 128: 1278 us unrolled, 1225 rolled; 64-wide heads with values of
// 128: 1077 and 1094; a cap alone 1165 and 1152).
template <int W>
__device__ __forceinline__ void stage_rows_bf16(uint32_t src, uint8_t* stage, int r, int wg, float mul, bool have,
                                                const float* add = nullptr, int n_add = 1, size_t add_stride = 0,
                                                bool all = false) {
  constexpr int HALF = W / 2;
#pragma unroll 1
  for (int c = 0; c < HALF / 32; ++c) {
    uint32_t v[32];
    if (have && !all) {
      tmem_ld32(src + c * 32, v);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = 0u;
    }
#pragma unroll 1
    for (int n = 0; add && n < n_add; ++n) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float4 a = __ldcg(reinterpret_cast<const float4*>(add + n * add_stride + c * 32) + q);
        v[4 * q] = __float_as_uint(__uint_as_float(v[4 * q]) + a.x);
        v[4 * q + 1] = __float_as_uint(__uint_as_float(v[4 * q + 1]) + a.y);
        v[4 * q + 2] = __float_as_uint(__uint_as_float(v[4 * q + 2]) + a.z);
        v[4 * q + 3] = __float_as_uint(__uint_as_float(v[4 * q + 3]) + a.w);
      }
    }
    const int col0 = wg * HALF + c * 32;  // first column of this chunk
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_bf16x2(__uint_as_float(v[8 * q + 2 * e]) * mul, __uint_as_float(v[8 * q + 2 * e + 1]) * mul);
      const int col = col0 + 8 * q;
      st_shared_v4(smem_u32(stage + (col >> 6) * (BN * 128) + sw128_offset(r, (col & 63) >> 3)), w[0], w[1], w[2],
                   w[3]);
    }
  }
}

// This row's fp32 sums of one accumulator (W columns in TMEM at src, this
// warpgroup's half of them) into a split item's partial area (zeros if the
// half saw no tile).
template <int W>
__device__ __forceinline__ void write_partial(uint32_t src, float* dst, bool have) {
  constexpr int HALF = W / 2;
#pragma unroll 1
  for (int c = 0; c < HALF / 32; ++c) {
    uint32_t v[32];
    if (have) {
      tmem_ld32(src + c * 32, v);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = 0u;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      __stcg(reinterpret_cast<float4*>(dst + c * 32) + q,
             make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                         __uint_as_float(v[4 * q + 3])));
  }
}

using fa::BwdParams;
using fa::ScoredBwdParams;
__device__ __forceinline__ bool parts_first(const BwdParams&) { return false; }
__device__ __forceinline__ bool parts_first(const ScoredBwdParams& p) { return p.split_first != 0; }
template <int SCORE>
using BwdParamsOf = std::conditional_t<SCORE >= 0, ScoredBwdParams, BwdParams>;

// The exponentials of 32 queries' scores of one key: raw q.k in sr -> fp32 weights
// for dS in pr (with a cap times a quarter of its derivative) and P as packed
// bf16.  lse: the queries' row statistics (log2 units); rel0: position of the
// first query minus the key's; vis: the queries that see the key (MASKED).
// BOTH: queries on both sides of the key may see it, else the bias is a line.
// SMALL: the cap by its polynomial; then returns whether every score was inside it.
template <bool CAP, bool SLOPES, bool MASKED, bool BOTH, bool SMALL>
__device__ __forceinline__ bool modified_chunk(const ScoredBwdParams& p, const uint32_t (&sr)[32], const float4* lse,
                                               int rel0, float slope2, uint32_t vis, float* pr, uint32_t (&pk)[16]) {
  const float in = CAP ? p.cap.in : p.scale_log2, log2c = CAP && !SMALL ? p.cap.log2c : 0.f;
  const uint64_t in2 = f2_pack(in, in), m2cap2 = f2_pack(-2.f * p.cap.log2c, -2.f * p.cap.log2c);
  const float side = rel0 + 31 <= 0 ? slope2 : -slope2;  // bias per step of the query
  uint64_t step[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) step[k] = f2_pack((float)(2 * k) * side, (float)(2 * k + 1) * side);
  const float rel = (float)rel0;
  float top = 0.f;  // greatest s^2
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    const float4 l4 = ld_shared_f4(lse + (c >> 2));  // 16-byte broadcast: 4 columns
    const uint64_t l[2] = {f2_pack(l4.x, l4.y), f2_pack(l4.z, l4.w)};
    uint64_t x[2] = {f2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])),
                     f2_pack(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]))};
    uint64_t r[2], e[2];
    if (CAP && !SMALL) cap_quad<false>(f2_mul(x[0], in2), f2_mul(x[1], in2), r[0], r[1], e[0], e[1]);
    const float gb = fmaf(rel + (float)c, side, log2c);  // (the sum is exact)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint64_t bias;  // (cap +) distance bias - row statistic
      if (SLOPES && BOTH) {
        const float d0 = (float)(rel0 + c + 2 * h), d1 = (float)(rel0 + c + 2 * h + 1);
        bias = f2_sub(f2_pack(fmaf(fabsf(d0), -slope2, log2c), fmaf(fabsf(d1), -slope2, log2c)), l[h]);
      } else if (SLOPES) {
        bias = f2_sub(f2_add(step[h], f2_pack(gb, gb)), l[h]);
      } else if (CAP && !SMALL) {
        bias = f2_sub(f2_pack(log2c, log2c), l[h]);
      } else {
        bias = f2_neg(l[h]);
      }
      uint64_t w = 0ull;  // a quarter of the cap's derivative
      if (CAP && SMALL) {
        const uint64_t u = f2_mul(x[h], x[h]);
        top = fmax3(top, f2_lo(u), f2_hi(u));
        uint64_t t = f2_fma(u, f2_pack(p.cap.a[4], p.cap.a[4]), f2_pack(p.cap.a[3], p.cap.a[3]));
        t = f2_fma(u, t, f2_pack(p.cap.a[2], p.cap.a[2]));
        t = f2_fma(u, t, f2_pack(p.cap.a[1], p.cap.a[1]));
        t = f2_mul(x[h], f2_fma(u, t, f2_pack(p.cap.a[0], p.cap.a[0])));
        w = f2_fma(f2_mul(t, t), f2_pack(p.cap.slope, p.cap.slope), f2_pack(0.25f, 0.25f));
        x[h] = f2_add(t, bias);
      } else if (CAP) {
        x[h] = f2_fma(r[h], m2cap2, bias);
        w = f2_mul(f2_mul(e[h], r[h]), r[h]);
      } else {
        x[h] = f2_fma(x[h], in2, bias);
      }
      float v0 = ex2(f2_lo(x[h])), v1 = ex2(f2_hi(x[h]));
      if (MASKED) {
        if (!((vis >> (c + 2 * h)) & 1u)) v0 = 0.f;
        if (!((vis >> (c + 2 * h + 1)) & 1u)) v1 = 0.f;
      }
      pk[c / 2 + h] = pack_bf16x2(v0, v1);
      w = CAP ? f2_mul(f2_pack(v0, v1), w) : f2_pack(v0, v1);
      pr[c + 2 * h] = f2_lo(w);
      pr[c + 2 * h + 1] = f2_hi(w);
    }
  }
  return !CAP || !SMALL || !__any_sync(0xffffffffu, top > p.cap.small2);
}

// Bits [from, to] of 64.
__device__ __forceinline__ void interval_bits(int from, int to, uint32_t (&vis)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int lo = min(max(from - 32 * k, 0), 32), hi = min(max(to + 1 - 32 * k, 0), 32);
    vis[k] = (uint32_t)(((1ull << hi) - 1) & ~((1ull << lo) - 1));
  }
}

// Whether query row q sees key j by the plan's row intervals (and, where they
// are compared key by key, documents).
__device__ __forceinline__ bool row_sees(const ScoredBwdParams& p, int b, int q, int j) {
  const size_t at = (size_t)b * p.q_tiles * BM + q;
  bool see = j >= __ldg(p.plan.row_lo + at) && j < __ldg(p.plan.row_hi + at);
  if (see && fa::plan_flag(p.plan.by_key, b))
    see = __ldg(p.plan.q_doc + at) == __ldg(p.plan.k_doc + (size_t)b * p.kv_tiles * BN + j);
  return see;
}
__device__ __noinline__ void rows_that_see(const ScoredBwdParams& p, int b, int q0, int j, uint32_t (&vis)[2]) {
  for (int k = 0; k < 2; ++k) {
    uint32_t bits = 0u;
    for (int c = 0; c < 32; ++c) bits |= (uint32_t)row_sees(p, b, q0 + 32 * k + c, j) << c;
    vis[k] = bits;
  }
}

// WINDOW (causal only): the sliding-window terms are compiled in only where
// a window is set, so the plain causal and full masks keep their lean code.
// SCORE: kPlain, or the score-modified form (CAUSAL and WINDOW are then not used).
template <int HD, int HDV, bool CAUSAL, bool WINDOW, int SCORE>
__global__ void __launch_bounds__(kThreads, 1)
    fa_bwd_main(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                const __grid_constant__ CUtensorMap tmdK, const __grid_constant__ CUtensorMap tmdV,
                const __grid_constant__ CUtensorMap tmAcc, const BwdParamsOf<SCORE> p) {
  using C = BwdCfg<HD, HDV>;
  if constexpr (SCORE >= 0) grid_next();
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int NQ = C::NQ, NDO = C::NDO;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* kv_full = bars + 0;
  uint64_t* q_full = bars + 1;         // [NQ]
  uint64_t* q_empty = q_full + NQ;     // [NQ]
  uint64_t* do_full = q_empty + NQ;    // [NDO]
  uint64_t* do_empty = do_full + NDO;  // [NDO]
  uint64_t* s_full = do_empty + NDO;
  uint64_t* dp_full = s_full + 1;
  uint64_t* p_ready = s_full + 2;
  uint64_t* ds_ready = s_full + 3;
  uint64_t* dq_full = s_full + 4;
  uint64_t* dq_empty = s_full + 5;
  uint64_t* acc_done = s_full + 6;
  uint64_t* drain = s_full + 7;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile unsigned int* split_seen = reinterpret_cast<volatile unsigned int*>(tmem_slot + 2);  // parts counted before

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // One linear grid in super-batches of sb_groups (batch, kv head) groups;
  // within a super-batch the key tile is slowest: its groups' tile 0 runs
  // first, then tile 1, ...  Causal low key tiles see the most query rows, so
  // each super-batch runs heaviest-first and the next one's heavy CTAs fill
  // the SMs its light ones free, which keeps the tail short.  Only a few
  // groups' Q, dO and fp32 dQ accumulator are live at a time, so they stay in
  // L2.  (One group at a time keeps even less live, but its late heavy CTAs
  // make the causal step ~12% longer.)
  // Plain calls have split items only without a causal mask (equal-work items): a
  // short last round, in two halves; the causal instances compile none of their
  // code.  Scored calls have them there too, and where there are few items of any
  // mask: the first ones, in `parts` parts (fa::BwdParams).
  constexpr bool MODS = SCORE >= 0, CAP = MODS && (SCORE & fa::kCap), SLOPES = MODS && (SCORE & fa::kSlopes);
  constexpr bool SPLIT = MODS || !CAUSAL;
  int item = blockIdx.x, split = -1, half = 0;
  int parts = 2;
  if constexpr (MODS) parts = p.parts;
  if (MODS && parts_first(p)) {
    // (unequal work: the first items of the order in `parts` parts each, launched first)
    if (item < p.n_split * parts) {
      split = item / parts;
      half = item - split * parts;
      item = split;
    } else {
      item -= p.n_split * (parts - 1);
    }
  } else if (SPLIT && item >= p.n_whole) {
    split = (item - p.n_whole) >> 1;
    half = (item - p.n_whole) & 1;
    item = p.n_whole + split;
  }
  const int per_sb = p.sb_groups * p.kv_tiles;
  const int sb = item / per_sb;
  const int in_sb = item - sb * per_sb;
  int n = in_sb / p.sb_groups;  // key tile
  const int bkv = sb * p.sb_groups + (in_sb - n * p.sb_groups);
  const int b = bkv / p.Hkv, hk = bkv - b * p.Hkv;
  if constexpr (MODS) {  // a plan's heaviest key tiles first
    if (p.plan.m_beg) n = min(max(p.plan.key_order[(size_t)b * p.kv_tiles + n], 0), p.kv_tiles - 1);
  }
  const int k0 = n * BN;

  int m_begin = 0, m_end = p.q_tiles;
  if constexpr (MODS) {
    if (p.plan.m_beg) {
      m_begin = max(0, p.plan.m_beg[(size_t)b * p.kv_tiles + n]);
      m_end = min(p.q_tiles, p.plan.m_end[(size_t)b * p.kv_tiles + n]);
    } else {
      m_begin = min(p.q_tiles, max(0, k0 - p.hi_off + 1) / BM);  // first row that sees key k0
      const int last_row = min(k0 + BN, p.Tk) - 1 - p.lo_off;    // last row that sees the tile's last key
      m_end = last_row < 0 ? 0 : min(p.q_tiles, last_row / BM + 1);
    }
  } else if (CAUSAL) {
    const int first_row = k0 - p.causal_off;  // first query row that sees key k0
    m_begin = first_row <= 0 ? 0 : min(p.q_tiles, first_row / BM);
    if (WINDOW) {
      // last query row whose window reaches the tile's last key
      const long long last_row = (long long)k0 + BN - 1 - p.causal_off + p.window - 1;
      m_end = last_row < 0 ? 0 : (int)min((long long)p.q_tiles, last_row / BM + 1);
    }
  }
  const int n_m = max(0, m_end - m_begin);
  const int T_item = p.G * n_m;  // the item's tiles
  if constexpr (MODS) {
    if (split >= 0 && p.plan.m_beg) {
      // The launcher counts without the plan: an item of few tiles after all runs in
      // fewer parts, or whole (part 0), and the CTAs of the rest leave.
      parts = min(parts, max(1, T_item / fa::kPlannedPartTiles));
      if (half >= parts) return;
      if (parts == 1) split = -1;
    }
  }
  // this CTA's tiles: [t0, t0 + T) of the item's
  int t0 = split >= 0 && half ? T_item / 2 : 0;
  int T = split >= 0 ? (half ? T_item - T_item / 2 : T_item / 2) : T_item;
  if constexpr (MODS) {
    if (split >= 0) {
      t0 = (int)((long long)T_item * half / parts);
      T = (int)((long long)T_item * (half + 1) / parts) - t0;
    }
  }

  if (threadIdx.x == 0) {
    *abort_flag = (smem_u32(smem) & 1023u) ? 1 : 0;
    mbar_init(kv_full, 1);
    for (int s = 0; s < NQ; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int s = 0; s < NDO; ++s) {
      mbar_init(&do_full[s], 1);
      mbar_init(&do_empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_ready, 256);
    // with VOUCH the dQ warps arrive too, once the previous dQ tile is drained
    mbar_init(ds_ready, C::VOUCH ? 384 : 256);
    mbar_init(dq_full, 1);
    mbar_init(dq_empty, 128);
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool run = (*abort_flag == 0) && T > 0;
  // d = 128: the dQ warpgroup holds a whole 128-column dQ row in registers so
  // that it can release dQ's TMEM columns before staging it; it takes the
  // registers the producer / MMA warpgroup does not need (setmaxnreg at the
  // top of both roles).  The launch gives every thread kRegsLaunch registers
  // (the launcher checks this), and the shares add up to that total:
  // kRegsLow + kRegsHigh = 2 * kRegsLaunch.
  const uint32_t T_S = tmem, T_DP = tmem + 128, T_DV = tmem + 256, T_DK = tmem + 256 + HDV;
  // dQ shares dP^T's columns unless there is room for columns of its own
  // (d = 64: dK ends at 384 or 448); then dP^T(t+1) need not wait for dQ(t)'s
  // drain, only dQ(t+1) does.
  constexpr bool kOwnDQ = 256 + HDV + 2 * HD <= 512;
  const uint32_t T_DQ = kOwnDQ ? T_DK + HD : T_DP;

  if (warp < 4) {
    if (kSplitRegs<HD>) setmaxnreg_dec<kRegsLow>();
    if (warp == 0 && lane == 0 && run) {
      // ---------------------------------------------------------- producer
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmdO);
      mbar_arrive_expect_tx(kv_full, C::QK_TILE + C::VO_TILE);
#pragma unroll
      for (int cb = 0; cb < HD / 64; ++cb) tma_load_3d(smem + C::OFF_K + cb * BN * 128, &tmK, kv_full, cb * 64, k0, bkv);
#pragma unroll
      for (int cb = 0; cb < HDV / 64; ++cb) tma_load_3d(smem + C::OFF_V + cb * BN * 128, &tmV, kv_full, cb * 64, k0, bkv);
      int last_q[NQ], last_do[NDO];
      for (int s = 0; s < NQ; ++s) last_q[s] = -1;
      for (int s = 0; s < NDO; ++s) last_do[s] = -1;
      for (int t = 0; t < T; ++t) {
        const int st = t % NQ, u = t / NQ;
        const int g = (t0 + t) / n_m, m = m_begin + ((t0 + t) - g * n_m);
        const int bh = b * p.Hq + hk * p.G + g;
        if (!mbar_wait(&q_empty[st], (u & 1) ^ 1, abort_flag)) break;
        mbar_arrive_expect_tx(&q_full[st], C::QK_TILE + 1024);
#pragma unroll
        for (int cb = 0; cb < HD / 64; ++cb)
          tma_load_3d(smem + C::OFF_Q + st * C::QK_TILE + cb * BM * 128, &tmQ, &q_full[st], cb * 64, m * BM, bh);
        const long long row0 = (long long)bh * p.Tq_pad + (long long)m * BM;
        bulk_load(smem + C::OFF_LSE + st * 512, p.lse2 + row0, 512, &q_full[st]);
        bulk_load(smem + C::OFF_DELTA + st * 512, p.delta + row0, 512, &q_full[st]);
        last_q[st] = u;
        // A dO slot is refilled only once dV of the tile before is done: pull
        // the tile into L2 now so that its load later does not stall the dP MMA.
#pragma unroll
        for (int cb = 0; cb < HDV / 64; ++cb) tma_prefetch_l2_3d(&tmdO, cb * 64, m * BM, bh);
        const int so = t % NDO, uo = t / NDO;
        if (!mbar_wait(&do_empty[so], (uo & 1) ^ 1, abort_flag)) break;
#ifdef FA_TEST_HOOKS
        if (p.test_withhold_do) continue;
#endif
        mbar_arrive_expect_tx(&do_full[so], C::VO_TILE);
#pragma unroll
        for (int cb = 0; cb < HDV / 64; ++cb)
          tma_load_3d(smem + C::OFF_DO + so * C::VO_TILE + cb * BM * 128, &tmdO, &do_full[so], cb * 64, m * BM, bh);
        last_do[so] = uo;
      }
      mbar_wait_bounded(kv_full, 0);
      for (int s = 0; s < NQ; ++s)
        if (last_q[s] >= 0) mbar_wait_bounded(&q_full[s], last_q[s] & 1);
      for (int s = 0; s < NDO; ++s)
        if (last_do[s] >= 0) mbar_wait_bounded(&do_full[s], last_do[s] & 1);
    } else if (warp == 1 && lane == 0 && run) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t id_sdp = idesc_bf16(BN, BM, 0, 0);  // S^T, dP^T: M = keys, N = queries
      constexpr uint32_t id_dv = idesc_bf16(BN, HDV, 0, 1);  // dV: M = keys, N = dv, B MN-major
      constexpr uint32_t id_dk = idesc_bf16(BN, HD, 0, 1);   // dK: M = keys, N = d, B MN-major
      constexpr uint32_t id_q = idesc_bf16(BM, HD, 1, 1);    // dQ: M = queries (A MN-major), N = d
      const uint32_t k_base = smem_u32(smem + C::OFF_K), v_base = smem_u32(smem + C::OFF_V);
      const uint32_t ds_base = smem_u32(smem + C::OFF_DS);
      const uint64_t k_desc = desc_kmajor(k_base), v_desc = desc_kmajor(v_base);
      const uint64_t k_desc_mn = desc_mnmajor(k_base, BN * 128), ds_desc = desc_mnmajor(ds_base, BN * 128);
      // S^T(t) = K Q_t^T into T_S
      auto mma_s = [&](int t) {
        const uint64_t q_desc = desc_kmajor(smem_u32(smem + C::OFF_Q + (t % NQ) * C::QK_TILE));
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t step = (k >> 2) * (BM * 128) + (k & 3) * 32;
          mma_ss(T_S, desc_at(k_desc, step), desc_at(q_desc, step), id_sdp, k > 0 ? 1u : 0u);
        }
        mma_commit(s_full);
      };
      // Issue order per tile t: dP^T(t), dV(t), S^T(t+1), dK(t), dQ(t).  S^T(t+1)
      // overwrites the P^T(t) columns dV(t) reads, and dQ(t) (d = 128) the dS^T(t)
      // columns dK(t) reads; one thread's MMAs execute in issue order, so both
      // have been read by then.  With S^T(t+1) right behind dV(t), the
      // elementwise warps go from tile t's dS phase straight to tile t+1's P
      // phase while dK(t), dQ(t) and dP^T(t+1) run.
      // With VOUCH the thread checks only p_ready(t) and ds_ready(t) per tile
      // (and dO(0)): those barriers also stand for Q(t+1) (before S^T(t+1)),
      // for dO(t+1) and for the drain of dQ(t) (before dQ(t+1) and dP^T(t+1)),
      // so dK(t), dQ(t) and dP^T(t+1) go out as one run of MMAs.
      bool ok = mbar_wait(kv_full, 0, abort_flag) && mbar_wait(&q_full[0], 0, abort_flag);
      if (ok) {
        tc_fence_after();
        mma_s(0);
      }
      for (int t = 0; ok && t < T; ++t) {
        const int st = t % NQ, so = t % NDO;
        const uint32_t q_base = smem_u32(smem + C::OFF_Q + st * C::QK_TILE);
        const uint32_t do_base = smem_u32(smem + C::OFF_DO + so * C::VO_TILE);
        if ((!C::VOUCH || t == 0) && !mbar_wait(&do_full[so], (t / NDO) & 1, abort_flag)) { ok = false; break; }
        // dP^T shares its TMEM columns with dQ (d = 128): the previous tile's dQ must be drained
        if (!kOwnDQ && t > 0 && !mbar_wait(dq_empty, (t - 1) & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint64_t do_desc = desc_kmajor(do_base);
#pragma unroll
        for (int k = 0; k < HDV / 16; ++k) {
          const uint32_t step = (k >> 2) * (BM * 128) + (k & 3) * 32;
          mma_ss(T_DP, desc_at(v_desc, step), desc_at(do_desc, step), id_sdp, k > 0 ? 1u : 0u);
        }
        mma_commit(dp_full);
        if (!mbar_wait(p_ready, t & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        // P^T lives in TMEM as packed bf16 over S^T: query columns [0,64) at TMEM
        // columns [0,32), query columns [64,128) at [64,96) (each elementwise
        // warpgroup overwrote its own half of S^T).
        const uint64_t do_desc_mn = desc_mnmajor(do_base, BM * 128);
#pragma unroll
        for (int k = 0; k < BM / 16; ++k)
          mma_ts(T_DV, T_S + (k >> 2) * 64 + (k & 3) * 8, desc_at(do_desc_mn, k * 2048), id_dv,
                 (t > 0 || k > 0) ? 1u : 0u);
        mma_commit(&do_empty[so]);
        if (t + 1 < T) {
          if (!C::VOUCH) {
            if (!mbar_wait(&q_full[(t + 1) % NQ], ((t + 1) / NQ) & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
          }
          mma_s(t + 1);
        }
        // dS^T lives in TMEM as packed bf16 over dP^T, in the same column
        // pattern as P^T: query columns [0,64) at [128,160), [64,128) at
        // [192,224).  (dK waits for all of it: by the time S^T(t+1) is
        // queued the elementwise warps have finished both halves, and every
        // extra barrier check would leave the tensor pipe idle for a
        // shared-memory round trip.)
        if (!mbar_wait(ds_ready, t & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint64_t q_desc_mn = desc_mnmajor(q_base, BM * 128);
#pragma unroll
        for (int k = 0; k < BM / 16; ++k)
          mma_ts(T_DK, T_DP + (k >> 2) * 64 + (k & 3) * 8, desc_at(q_desc_mn, k * 2048), id_dk,
                 (t > 0 || k > 0) ? 1u : 0u);
        mma_commit(&q_empty[st]);
        if (kOwnDQ && !C::VOUCH && t > 0) {  // dQ(t-1) drained from its columns
          if (!mbar_wait(dq_empty, (t - 1) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
        }
#pragma unroll
        for (int k = 0; k < BN / 16; ++k)
          mma_ss(T_DQ, desc_at(ds_desc, k * 2048), desc_at(k_desc_mn, k * 2048), id_q,
                 k > 0 ? 1u : 0u);
        mma_commit(dq_full);
      }
      mma_commit(acc_done);
      mma_commit(drain);
      mbar_wait_bounded(drain, 0);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ elementwise warpgroups
    const int wg = (warp - 4) >> 2;  // 0 or 1
    const int quad = warp & 3;
    const int r = quad * 32 + lane;  // TMEM lane = key row
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const int key = k0 + r;
    const bool key_valid = key < p.Tk;
    const float sl2 = p.scale_log2;
    int row_from = 0x40000000, row_to = 0;  // query rows that see this key (MODS)
    bool by_row = false;                    // look each row's interval up instead
    if constexpr (MODS) {
      if (p.plan.m_beg) {
        const size_t at = (size_t)b * p.kv_tiles * BN + key;
        row_from = p.plan.key_from[at];
        row_to = p.plan.key_to[at] - 1;
        by_row = fa::plan_flag(p.plan.by_row, b);
      } else if (key_valid) {
        row_from = key - p.hi_off + 1;
        row_to = key - p.lo_off;
      }
    }
    bool ok = run;
    // With VOUCH one thread checks the next tile's Q before releasing P and
    // its dO before releasing dS, standing in for the MMA thread's checks.
    const bool voucher = C::VOUCH && warp == 4 && lane == 0;
    for (int t = 0; ok && t < T; ++t) {
      const int st = t % NQ, u = t / NQ;
      const int g = (t0 + t) / n_m, m = m_begin + ((t0 + t) - g * n_m);
      const int q0 = m * BM;
      const float* lse_s = reinterpret_cast<const float*>(smem + C::OFF_LSE + st * 512);
      const float* del_s = reinterpret_cast<const float*>(smem + C::OFF_DELTA + st * 512);
      // Each warp agrees on the outcome of the waits before its collective
      // TMEM loads and stores, so a timeout never splits a warp.
      bool got = mbar_wait(&q_full[st], u & 1, abort_flag) && mbar_wait(s_full, t & 1, abort_flag);
      if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
      tc_fence_after();
      // ---- P = exp2(S * scale * log2e - L2), masked; 32 query columns at a time.
      // The packed bf16 P of chunk c is stored over S columns this thread has
      // already read (each thread only touches its own TMEM lane); the fp32 P
      // stays in registers for dS.
      const float4* lse4 = reinterpret_cast<const float4*>(lse_s + wg * 64);
      const uint64_t sl2x2 = f2_pack(sl2, sl2);
      float pr[64];
      if constexpr (MODS) {
        // which of this warpgroup's 64 queries see this thread's key, by bits
        const int c0 = q0 + wg * 64;  // first of them
        uint32_t vis[2] = {~0u, ~0u};
        const int rel0 = c0 + p.causal_off - key;  // of query c0 to the key
        // (chunks that cross the key's position go with the masked ones: they are rare)
        const bool masked = by_row || __any_sync(0xffffffffu, row_from > c0 || row_to < c0 + 63 ||
                                                                  (SLOPES && p.two_sided && rel0 < 0 && rel0 + 64 > 1));
        if (masked) {
          if (by_row)
            rows_that_see(p, b, c0, key, vis);
          else
            interval_bits(row_from - c0, row_to - c0, vis);
        }
        float slope2 = 0.f;
        if (SLOPES) slope2 = p.slopes[hk * p.G + g] * 1.4426950408889634f;
        auto chunk = [&](auto ch_, auto masked_) {
          constexpr int ch = decltype(ch_)::value;
          uint32_t sr[32], pk[16];
          tmem_ld32(T_S + lane_base + wg * 64 + ch * 32, sr);
          tmem_wait_ld();
          constexpr bool M = decltype(masked_)::value, B = M && SLOPES;
          // (with slopes the masked chunks go by the general form alone: less code and
          // fewer registers, 1322 -> 1283 us at T 8192, 32 heads of 128)
          if (!modified_chunk<CAP, SLOPES, M, B, CAP && !(SLOPES && M)>(p, sr, lse4 + ch * 8, rel0 + ch * 32, slope2, vis[ch],
                                                      pr + ch * 32, pk)) {
            // a score past the polynomial: the whole chunk again (its scores are still in TMEM)
            tmem_ld32(T_S + lane_base + wg * 64 + ch * 32, sr);
            tmem_wait_ld();
            modified_chunk<CAP, SLOPES, M, B, false>(p, sr, lse4 + ch * 8, rel0 + ch * 32, slope2, vis[ch],
                                                     pr + ch * 32, pk);
          }
          tmem_st16(T_S + lane_base + wg * 64 + ch * 16, pk);
        };
        using zero = std::integral_constant<int, 0>;
        using one = std::integral_constant<int, 1>;
        if (!masked) {
          chunk(zero{}, std::false_type{});
          chunk(one{}, std::false_type{});
        } else {
          chunk(zero{}, std::true_type{});
          chunk(one{}, std::true_type{});
        }
      } else {
        const bool need_mask = !key_valid || (CAUSAL && k0 + BN - 1 > q0 + p.causal_off) ||
                               (WINDOW && q0 + BM - 1 + p.causal_off - p.window + 1 > k0);
        // key row `key` is visible to query q0 + c iff vis_from <= c <= vis_to:
        // key <= q0 + c + off, and with a window also key > q0 + c + off - W
        const int vis_from = key_valid ? (CAUSAL ? key - p.causal_off - q0 : -0x40000000) : 0x40000000;
        const int vis_to = WINDOW ? key - p.causal_off - q0 + p.window - 1 : 0x40000000;
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t sr[32];
          tmem_ld32(T_S + lane_base + wg * 64 + ch * 32, sr);
          tmem_wait_ld();
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 l4 = ld_shared_f4(lse4 + ((ch * 32 + c) >> 2));  // 16-byte broadcast: 4 columns
            const uint64_t x01 = f2_fma(f2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sl2x2,
                                        f2_pack(-l4.x, -l4.y));
            const uint64_t x23 = f2_fma(f2_pack(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3])), sl2x2,
                                        f2_pack(-l4.z, -l4.w));
            float v0 = ex2(f2_lo(x01)), v1 = ex2(f2_hi(x01)), v2 = ex2(f2_lo(x23)), v3 = ex2(f2_hi(x23));
            if (need_mask) {
              const int qc = wg * 64 + ch * 32 + c;
              if (qc < vis_from || (WINDOW && qc > vis_to)) v0 = 0.f;
              if (qc + 1 < vis_from || (WINDOW && qc + 1 > vis_to)) v1 = 0.f;
              if (qc + 2 < vis_from || (WINDOW && qc + 2 > vis_to)) v2 = 0.f;
              if (qc + 3 < vis_from || (WINDOW && qc + 3 > vis_to)) v3 = 0.f;
            }
            pr[ch * 32 + c] = v0;
            pr[ch * 32 + c + 1] = v1;
            pr[ch * 32 + c + 2] = v2;
            pr[ch * 32 + c + 3] = v3;
            pk[c / 2] = pack_bf16x2(v0, v1);
            pk[c / 2 + 1] = pack_bf16x2(v2, v3);
          }
          tmem_st16(T_S + lane_base + wg * 64 + ch * 16, pk);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      if (voucher && t + 1 < T && !mbar_wait(&q_full[(t + 1) % NQ], ((t + 1) / NQ) & 1, abort_flag)) ok = false;
      mbar_arrive(p_ready);
      if (C::VOUCH && !__all_sync(0xffffffffu, ok)) { ok = false; break; }  // the warp stops as one
      // ---- dS = P * (dP - D) -> shared memory (row = key, 128B-swizzled, query-contiguous)
      // dP^T is in TMEM.  The previous tile's dQ MMA, which reads dS from shared
      // memory, was issued before this tile's dP^T by the same thread, so the
      // dP^T commit covers it too.
      got = mbar_wait(dp_full, t & 1, abort_flag);
      if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
      tc_fence_after();
      uint8_t* ds_blk = smem + C::OFF_DS + wg * (BN * 128);
      const float4* del4 = reinterpret_cast<const float4*>(del_s + wg * 64);
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t dr[32];
        tmem_ld32(T_DP + lane_base + wg * 64 + ch * 32, dr);
        tmem_wait_ld();
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const int c = cc * 8 + 2 * e;  // column inside the chunk (4 per step)
            const float4 d4 = ld_shared_f4(del4 + ((ch * 32 + c) >> 2));
            const uint64_t g01 = f2_sub(f2_pack(__uint_as_float(dr[c]), __uint_as_float(dr[c + 1])), f2_pack(d4.x, d4.y));
            const uint64_t g23 = f2_sub(f2_pack(__uint_as_float(dr[c + 2]), __uint_as_float(dr[c + 3])), f2_pack(d4.z, d4.w));
            const uint64_t s01 = f2_mul(g01, f2_pack(pr[ch * 32 + c], pr[ch * 32 + c + 1]));
            const uint64_t s23 = f2_mul(g23, f2_pack(pr[ch * 32 + c + 2], pr[ch * 32 + c + 3]));
            w[e] = pack_bf16x2(f2_lo(s01), f2_hi(s01));
            w[e + 1] = pack_bf16x2(f2_lo(s23), f2_hi(s23));
          }
          st_shared_v4(smem_u32(ds_blk + sw128_offset(r, ch * 4 + cc)), w[0], w[1], w[2], w[3]);
          // packed dS^T of these 8 columns, for the dK MMA (A from TMEM), over
          // dP^T columns this thread has already read
          tmem_st4(T_DP + lane_base + wg * 64 + ch * 16 + cc * 4, w[0], w[1], w[2], w[3]);
        }
      }
      tmem_wait_st();
      fence_async_smem();
      tc_fence_before();
      if (voucher && t + 1 < T && !mbar_wait(&do_full[(t + 1) % NDO], ((t + 1) / NDO) & 1, abort_flag)) ok = false;
      mbar_arrive(ds_ready);
      if (C::VOUCH && !__all_sync(0xffffffffu, ok)) { ok = false; break; }
    }
    // ---- epilogue: dV, dK * scale -> bf16 -> shared (the Q ring, idle now) -> TMA store
    if (ok && T > 0) {
      if (!__all_sync(0xffffffffu, mbar_wait(acc_done, 0, abort_flag))) ok = false;
      tc_fence_after();
    }
    const bool mine = (T == 0 || ok) && *abort_flag == 0;
    if (named_bar_and(1, 256, mine)) {
      // A split item's parts (or halves): each writes its fp32 sums to the partial
      // area and counts itself in; the one that comes last adds the others' sums and
      // its own and stores the item's dV and dK.  None waits for another.
      const float* other = nullptr;
      bool finish = true;
      size_t slot0 = (size_t)split * 2;  // the item's first slot of the partial area
      if constexpr (MODS) slot0 = (size_t)split * p.parts;
      if (split >= 0) {
        // (modified scores: the half that finds the other counted in is the last, and
        // need not write its own sums)
        bool last = false;
        if (MODS && parts == 2) {
          if (warp == 4 && lane == 0) *split_seen = __ldcg(&p.split_counters[split]);
          named_bar_sync(3, 256);
          last = *split_seen == 1u;
          named_bar_sync(3, 256);  // all have read it
        }
        if (last) {
          finish = true;
        } else {
          float* own = p.part + ((slot0 + half) * BN + r) * (HD + HDV);
          write_partial<HDV>(T_DV + lane_base + wg * (HDV / 2), own + wg * (HDV / 2), T > 0);
          write_partial<HD>(T_DK + lane_base + wg * (HD / 2), own + HDV + wg * (HD / 2), T > 0);
          __threadfence();
          named_bar_sync(3, 256);
          if (warp == 4 && lane == 0) *split_seen = atomicAdd(&p.split_counters[split], 1u);
          named_bar_sync(3, 256);
          finish = *split_seen == (unsigned)parts - 1u;
        }
        if (finish) {
          __threadfence();
          other = p.part + (slot0 * BN + r) * (HD + HDV);
          if (parts == 2) other += (size_t)(half ^ 1) * BN * (HD + HDV);
        }
      }
      // (two sums are the same in either order)
      const bool all = parts > 2 && other;
      const int n_other = all ? parts : 1;
      constexpr size_t kPartStride = (size_t)BN * (HD + HDV);
      if (!finish) goto epilogue_done;
      stage_rows_bf16<HDV>(T_DV + lane_base + wg * (HDV / 2), smem + C::OFF_DV_STAGE, r, wg, 1.f, T > 0,
                           other ? other + wg * (HDV / 2) : nullptr, n_other, kPartStride, all);
      stage_rows_bf16<HD>(T_DK + lane_base + wg * (HD / 2), smem + C::OFF_DK_STAGE, r, wg, p.scale_grad, T > 0,
                          other ? other + HDV + wg * (HD / 2) : nullptr, n_other, kPartStride, all);
      fence_async_smem();
      named_bar_sync(2, 256);
      if (warp == 4 && lane == 0) {
        prefetch_tmap(&tmdV);
        prefetch_tmap(&tmdK);
#pragma unroll
        for (int cb = 0; cb < HDV / 64; ++cb)
          tma_store_3d(&tmdV, smem + C::OFF_DV_STAGE + cb * BN * 128, cb * 64, k0, bkv);
#pragma unroll
        for (int cb = 0; cb < HD / 64; ++cb)
          tma_store_3d(&tmdK, smem + C::OFF_DK_STAGE + cb * BN * 128, cb * 64, k0, bkv);
        bulk_commit();
        bulk_wait0();
      }
    }
  epilogue_done:;
  } else {
    // ------------------------------------------------------------ dQ warpgroup
    if (kSplitRegs<HD>) setmaxnreg_inc<kRegsHigh>();
    // Each warp drains its own 32 query rows (its TMEM lanes).  It copies all
    // of its rows of dQ_t out of TMEM first and releases the columns at once
    // (dP^T of the next tile waits for them at d = 128), then adds them into
    // the fp32 accumulator two 32-column chunks at a time: two 4 KB staging
    // slots per warp (32 rows x 32 fp32, 128B-swizzled), one 32x32 TMA
    // reduce-add per slot; only warp-local ordering is needed.
    const int quad = warp & 3;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const bool leader = (lane == 0);
    uint8_t* wslot = smem + C::OFF_STG + quad * (2 * C::STG_SLOT);
    constexpr int NCH = HD / 32;  // 32-column chunks per tile
    bool ok = run;
    // With VOUCH the drain is announced on ds_ready(t+1) (which the MMA thread
    // waits for before dQ(t+1) anyway); there is nothing to drain before dQ(0).
    if (C::VOUCH && ok) mbar_arrive(ds_ready);
    for (int t = 0; ok && t < T; ++t) {
      const int g = (t0 + t) / n_m, m = m_begin + ((t0 + t) - g * n_m);
      const int bh = b * p.Hq + hk * p.G + g;
      if (!__all_sync(0xffffffffu, mbar_wait(dq_full, t & 1, abort_flag))) { ok = false; break; }
      tc_fence_after();
      uint32_t v[NCH][32];
#pragma unroll
      for (int c = 0; c < NCH; ++c) tmem_ld32(T_DQ + lane_base + c * 32, v[c]);
      tmem_wait_ld();
      tc_fence_before();
      // all of dQ_t is out of TMEM: it may take dP_{t+1} (or dQ_{t+1})
      if (!C::VOUCH)
        mbar_arrive(dq_empty);
      else if (t + 1 < T)
        mbar_arrive(ds_ready);
#pragma unroll
      for (int c = 0; c < NCH; c += 2) {
        if (leader) bulk_wait_read0();  // both slots read by the previous reduce-adds
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          st_shared_v4(smem_u32(wslot + sw128_offset(lane, q)), v[c][4 * q], v[c][4 * q + 1], v[c][4 * q + 2],
                       v[c][4 * q + 3]);
          st_shared_v4(smem_u32(wslot + C::STG_SLOT + sw128_offset(lane, q)), v[c + 1][4 * q], v[c + 1][4 * q + 1],
                       v[c + 1][4 * q + 2], v[c + 1][4 * q + 3]);
        }
        fence_async_smem();
        __syncwarp();
        if (leader) {
          tma_reduce_add_3d(&tmAcc, wslot, c * 32, m * BM + quad * 32, bh);
          tma_reduce_add_3d(&tmAcc, wslot + C::STG_SLOT, (c + 1) * 32, m * BM + quad * 32, bh);
          bulk_commit();
        }
      }
    }
    if (leader) bulk_wait0();  // every reduce-add has landed before the kernel ends
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicExch(p.status, DEV_TIMEOUT);
}

template <int HD, int HDV, bool CAUSAL, bool WINDOW, int SCORE>
cudaError_t launch_main_t(const fa::Problem& pr, const CUtensorMap* maps, const BwdParamsOf<SCORE>& bp,
                          cudaStream_t stream) {
  using C = BwdCfg<HD, HDV>;
  const void* fn = reinterpret_cast<const void*>(fa_bwd_main<HD, HDV, CAUSAL, WINDOW, SCORE>);
  cudaError_t e = fa::allow_dynamic_smem(fn, C::SMEM);
  if (e != cudaSuccess) return e;
  if (kSplitRegs<HD>) {
    // The register split only balances if every thread was launched with
    // exactly kRegsLaunch registers; otherwise the dQ warpgroup's request
    // could never be met, so refuse to launch.
    cudaFuncAttributes fa_attr;
    e = cudaFuncGetAttributes(&fa_attr, fn);
    if (e != cudaSuccess) return e;
    if (fa_attr.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
  }
  // one CTA per item, two (or `parts`) per split item (within int range: checked by the API, n_split <= kMaxSplitItems)
  int parts = 2;
  if constexpr (SCORE >= 0) parts = bp.parts;
  dim3 grid((unsigned)(bp.n_whole + parts * bp.n_split));
  fa_bwd_main<HD, HDV, CAUSAL, WINDOW, SCORE><<<grid, kThreads, C::SMEM, stream>>>(maps[0], maps[1], maps[2], maps[3], maps[4], maps[5],
                                                               maps[6], bp);
  return cudaGetLastError();
}

}  // namespace
