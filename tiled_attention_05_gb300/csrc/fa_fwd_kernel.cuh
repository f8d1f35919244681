// Forward kernel of tiled exact attention on sm_103a (the plain instances are
// in fa_fwd.cu, the score-modified ones in fa_scored_fwd_*.cu).
//
// Method ("What Ordinary Autograd Saves: Tiling the Forward Pass Is Only Half
// the Algorithm", section "The implementation under test"): for one block of
// query rows, walk the key/value blocks keeping per row a running maximum m,
// a running sum of exponentials l and an unnormalised output; rescale the
// output when the maximum moves; normalise once at the end and emit
// L = m + log(l) beside O.  Nothing of size Tq x Tk is ever stored.
//
// GB300 mapping: a persistent grid of one CTA per SM.  A work item is two
// 128-row query tiles (A and B) of one (batch, head), sharing every K/V tile
// the CTA loads for it; each CTA walks its items (heaviest causal rows first,
// in a snake order over the CTAs so that their totals even out) and starts
// the next item's loads and first MMAs while the current one finishes.
// Without a causal mask (items of equal work) a last round with at most half
// as many items as SMs is run as single-tile items (tile B left empty) on
// twice as many SMs.
//   warp 0       TMA producer: Q_A, Q_B per item (each as soon as the last
//                S of the previous item's tile has read its buffer), then the
//                item's K_j / V_j through NS-deep rings that run on across items.
//   warp 1       tcgen05 issuer.  Per key tile j it issues, in this order,
//                  O_A += P_A(j) V_j,  S_A(j+1) = Q_A K_{j+1}^T,
//                  O_B += P_B(j) V_j,  S_B(j+1) = Q_B K_{j+1}^T,
//                so while one softmax warpgroup works on its tile the tensor
//                pipe runs the other tile's two MMAs (ping-pong).  P is read
//                straight from TMEM (A operand); the MMAs of one thread execute
//                in issue order, so S_X(j+1) overwrites P_X(j) only after the
//                P.V that reads it.  An item's first S MMAs follow the previous
//                item's last P.V at once, while the softmax warpgroups write
//                that item's output.
//   warps 4..7   softmax of tile A, warps 8..11 softmax of tile B (thread =
//                query row = TMEM lane): load the score row, mask, row max,
//                exp2, row sum, write P as packed bf16 over the scores in TMEM;
//                rescale the O row in TMEM when the max grows by more than 2^8
//                (lazy rescaling, exact after the final normalisation);
//                epilogue O / l -> bf16 -> global (each thread its row), L -> global.
//                The next item's first P.V into O_X waits for this warpgroup's
//                first P of that item, which it writes only after its epilogue
//                has read O_X out of TMEM.
//                The two softmax warpgroups take registers from the producer /
//                MMA warpgroup (setmaxnreg), so that a whole score row stays in
//                registers without spilling.
// TMEM columns: S_A/P_A [0,128), S_B/P_B [128,256), O_A [256,256+dv), O_B [384,384+dv).
// Scores are kept in log2 units (scale * log2(e) folded into one FMA).
//
// Each tile visits the key tiles [beg, end) its rows can see (causal: up to
// the diagonal; with a sliding window of W keys also from the first row's
// window start on).  The CTA loads the union of the two ranges once; a key
// tile inside the union that one tile does not need is skipped by that tile's
// MMAs and softmax.  Every barrier phase (and ring position) is counted from
// the start of the CTA, not of the item.
//
// Score-modified instances (SCORE >= 0; bits in fa::ScoreBits) change the scores
// between their TMEM load and the exponential, in log2 units:
//   cap     x = c tanh(s / c) = c - 2 c / (1 + exp(2 s / c)): one ex2, a quarter of a
//           reciprocal (cap_quad) and one FMA per element, off by at most 2^-20 of c
//           (the single-instruction tanh is good to 2^-11 only, which would put
//           0.02 on a score near a cap of 50); an odd polynomial where |s| <= c / 2.
//   slopes  x -= slope_h |i + Tk - Tq - j|: a line in the column on either side of
//           the row's position, which joins the exponent.
// kBounded: a capped score is bounded, so no maximum is looked for and O is never
// rescaled (bounded_tile).  kSlopes alone: two passes over the scores in TMEM
// (line_max, line_exp).  The rest holds a row in registers as the plain form does.
// Their masks are one interval of keys per row, [lo, hi): causal, window and
// tail are lines in i, documents and prefixes come from a mask plan (see
// fa_mask_plan.cu), which also holds each query tile's key-tile range.  A warp
// masks a tile only where one of its rows does not see all of it.
// What bounds them is the MMA-issuing thread, as in the plain form, and beside it
// the softmax: the more its warps issue, the longer each group of MMAs takes to
// issue (PV 602 cycles a group plain, 731 with a cap, 774 with both; the softmax
// 1050, 1800 and 2100 cycles a tile).  B 2, 32 / 8 heads of 128, T 8192, causal:
// 758 us plain, 960 with a cap of 50 or slopes, 1060 with both; 1249 with a cap whose half
// the scores pass; 4 batches of 16 heads of 64, T 2048: 54, 78 with a cap (98 past its
// half), 74 and 85.
#pragma once
#include <cstdint>
#include <type_traits>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

using namespace fa_ptx;

namespace {

constexpr int BM = fa::kTile;  // query rows per tile (two tiles per work item)
constexpr int BN = fa::kTile;  // keys per tile
constexpr int kThreads = 384;
// Register split: every thread starts with kRegsLaunch; the producer / MMA
// warpgroup drops to kRegsLow and the two softmax warpgroups rise to
// kRegsHigh (one score row of 128 fp32 values and its packed P in registers
// without spilling).  kRegsLow + 2 * kRegsHigh = 3 * kRegsLaunch.
constexpr int kRegsLaunch = 168;  // 65536 / 384 rounded down to a multiple of 8
constexpr int kRegsLow = 88;
constexpr int kRegsHigh = (3 * kRegsLaunch - kRegsLow) / 2;  // 208
static_assert(kRegsLow + 2 * kRegsHigh == 3 * kRegsLaunch && kRegsHigh % 8 == 0, "setmaxnreg operands");
constexpr float kRescaleThreshold = 8.0f;  // log2 units: P stays <= 256 between rescales

// The forward's waits: mbar_wait with a suspend-time hint on try_wait.  A
// thread that finds the phase incomplete then sleeps until it completes (or
// the hint runs out) and is woken ~80 cycles after the completing arrival,
// against 100-160 with the default limit (measured).  Same bounds and abort
// behaviour as mbar_wait.
constexpr uint32_t kSuspendHintNs = 100000u;
__device__ __forceinline__ bool try_wait_hinted(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendHintNs)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool fwd_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         uint64_t timeout_ns = 2000000000ull) {
  if (try_wait_hinted(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  uint32_t spins = 0;
  while (true) {
    if (try_wait_hinted(bar, parity)) return true;
    if ((++spins & 63u) == 0) {
      if (*abort) return false;
      if (globaltimer_ns() - t0 > timeout_ns) {
        *abort = 1;
        return false;
      }
    }
  }
}

// HD: head size of Q and K (the score contraction); HDV: head size of V and O.
template <int HD, int HDV>
struct FwdCfg {
  static constexpr int NS = (HD == 64 && HDV == 64) ? 4 : 2;  // K/V ring depth
  // With a 4-deep ring K_{j+1} / V_{j+1} have landed long before tile j's P is
  // ready, so the softmax checks them and the MMA thread saves a barrier
  // check per key tile.  With a 2-deep ring they often land later than that,
  // and tying P_X(j).V to them would stall the tensor pipe.
  static constexpr bool KV_VIA_SOFTMAX = NS >= 3;
  static constexpr int Q_BYTES = BM * HD * 2;
  static constexpr int K_BYTES = BN * HD * 2;
  static constexpr int V_BYTES = BN * HDV * 2;
  static constexpr int OFF_Q = 0;  // [2]: tile A, tile B
  static constexpr int OFF_K = OFF_Q + 2 * Q_BYTES;
  static constexpr int OFF_V = OFF_K + NS * K_BYTES;
  static constexpr int OFF_BAR = OFF_V + NS * V_BYTES;
  static constexpr int NBAR = 2 + 2 + 3 * NS + 2 + 2 + 2 + 1;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct FwdParams {
  uint16_t* O;  // bf16 [B, Hq, Tq, dv]
  float* L;
  int* status;
  int Hq, Hkv, G, Tq, Tk;
  int causal_off;  // Tk - Tq
  int window;      // causal sliding window in keys, 0 = none
  int kv_tiles;
  int n_bh;            // B * Hq
  int n_pairs;         // query-tile pairs per (batch, head)
  long long n_full;    // work items that are pairs of query tiles
  long long n_items;   // all work items: n_full pairs, then single query tiles
  float scale_log2;  // scale * log2(e)
  int test_withhold_q;  // test build only: never issue the Q loads (every wait then times out)
};

// What the score-modified instances need besides (see fa::ScoreMods).
struct ScoredFwdParams : FwdParams {
  fa::CapParams cap;
  const float* slopes;  // [Hq]
  int hi_off, lo_off;   // row i sees keys [i + lo_off, i + hi_off) (no plan)
  int q_tiles;
  int two_sided;        // a row may see keys on both sides of its own position
  int row_mod, group;   // packed heads (fa::FwdShape)
  int split;            // CTAs per item
  float* part;          // [items][split][256 rows][dv], then as many (m, l, l of O, 0)
  fa::PlanView plan;
};
template <int SCORE>
constexpr bool kIsFew = SCORE >= 0 && (SCORE & fa::kFew) != 0;
template <int SCORE>
using FwdParamsOf = std::conditional_t<SCORE >= 0, ScoredFwdParams, FwdParams>;

// Key tiles [*beg, *end) that query rows [qa, qa+128) must visit (empty: 0, 0).
template <bool CAUSAL, bool WINDOW, int SCORE>
__device__ __forceinline__ void kv_range_for(const FwdParamsOf<SCORE>& p, int b, int qa, int* beg, int* end) {
  *beg = *end = 0;
  if (qa >= p.Tq) return;
  if constexpr (SCORE >= 0) {
    int bg, e;
    if (p.plan.kv_beg) {
      const size_t at = (size_t)b * p.q_tiles + (kIsFew<SCORE> && p.row_mod ? 0 : qa / BM);
      bg = max(0, p.plan.kv_beg[at]);
      e = min(p.kv_tiles, p.plan.kv_end[at]);
    } else {
      const bool packed = kIsFew<SCORE> && p.row_mod;
      const int first = packed ? 0 : qa, last = packed ? p.row_mod - 1 : min(qa + BM, p.Tq) - 1;  // positions
      const int hi = min(p.Tk, last + p.hi_off);  // keys the last row sees end here
      bg = max(0, first + p.lo_off) / BN;
      e = hi > 0 ? (hi + BN - 1) / BN : 0;
    }
    if (bg < e) {
      *beg = bg;
      *end = e;
    }
    return;
  }
  if (!CAUSAL) {
    *end = p.kv_tiles;
    return;
  }
  const int last_key = min(qa + BM, p.Tq) - 1 + p.causal_off;  // last key the tile's last row sees
  if (last_key < 0) return;
  const int e = min(p.kv_tiles, last_key / BN + 1);
  int bg = 0;
  if (WINDOW) {
    const int first_key = qa + p.causal_off - p.window + 1;  // first key the tile's first row sees
    bg = first_key > 0 ? first_key / BN : 0;
  }
  if (bg < e) {
    *beg = bg;
    *end = e;
  }
}

// One work item: query tiles A = [q0, q0 + 128) and B = [q0 + 128, q0 + 256)
// of (batch, head) bh, and the key tiles each must visit.
struct FwdItem {
  int bh, q0, bkv;
  int kb[2], ke[2];  // key-tile range of tile A and tile B
  int ub, ue;        // their union, loaded once
  bool single;       // tile B is not part of the item (its rows belong to another item)
};

// Index of the n-th item of this CTA (see fwd_item).
__device__ __forceinline__ long long fwd_index(int n) {
  const long long G = gridDim.x, c = blockIdx.x;
  return n * G + ((n & 1) ? G - 1 - c : c);
}

// The n-th item of this CTA, or false past its last.  Items are numbered
// heaviest causal rows first (the pair index slowest); round n of the grid
// takes items [n * G, n * G + G), CTA c the c-th of them in even rounds and
// the (G - 1 - c)-th in odd ones, so each CTA's heavy and light items pair up.
// Past n_full, every pair is split into two single-tile items (tile B empty),
// which spreads a short last round of equal-weight items over twice as many
// CTAs.
template <bool CAUSAL, bool WINDOW, int SCORE>
__device__ __forceinline__ bool fwd_item(const FwdParamsOf<SCORE>& p, int n, FwdItem* it) {
  long long k = fwd_index(n);
  if (k >= p.n_items) return false;
  int share = 0;
  if constexpr (kIsFew<SCORE>) {
    if (p.split > 1) {
      share = (int)(k % p.split);
      k /= p.split;
    }
  }
  const bool single = k >= p.n_full;
  it->single = single;
  const long long kp = single ? p.n_full + ((k - p.n_full) >> 1) : k;  // the pair
  int y = (int)(kp / p.n_bh);
  it->bh = (int)(kp - (long long)y * p.n_bh);
  const int b = it->bh / p.Hq, h = it->bh - b * p.Hq;
  y = p.n_pairs - 1 - y;
  if constexpr (SCORE >= 0) {  // a plan's heaviest pairs first (the parts of split items go by position)
    if (p.plan.kv_beg && (!kIsFew<SCORE> || (!p.row_mod && p.split == 1)))
      y = min(max(p.plan.pair_order[(size_t)b * p.n_pairs + p.n_pairs - 1 - y], 0), p.n_pairs - 1);
  }
  it->q0 = y * (2 * BM) + (single ? (int)((k - p.n_full) & 1) * BM : 0);
  it->bkv = b * p.Hkv + h / p.G;
  kv_range_for<CAUSAL, WINDOW, SCORE>(p, b, it->q0, &it->kb[0], &it->ke[0]);
  if (single) {
    it->kb[1] = it->ke[1] = 0;
  } else {
    kv_range_for<CAUSAL, WINDOW, SCORE>(p, b, it->q0 + BM, &it->kb[1], &it->ke[1]);
  }
  // Tile B's rows follow tile A's, so B's range starts and ends no earlier
  // than A's, and starts no later than A's end: the union has no gap and
  // every key tile in it is needed by A or B.
  it->ub = it->ke[0] > it->kb[0] ? it->kb[0] : it->kb[1];
  it->ue = max(it->ke[0], it->ke[1]);
  // A plan's ranges are any two: the earlier one is stretched over a gap
  // between them (its extra tiles are masked whole), because a key tile that
  // neither tile visits would never be released.
  if constexpr (SCORE >= 0) {
    if (it->ke[0] > it->kb[0] && it->ke[1] > it->kb[1]) {
      if (it->ke[0] < it->kb[1]) it->ke[0] = it->kb[1];
      if (it->ke[1] < it->kb[0]) it->ke[1] = it->kb[0];
      it->ub = min(it->kb[0], it->kb[1]);
    }
    if (kIsFew<SCORE> && p.split > 1) {  // this CTA's share of the key tiles
      const int len = (it->ue - it->ub + p.split - 1) / p.split;
      const int from = min(it->ub + share * len, it->ue), to = min(from + len, it->ue);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        it->kb[x] = max(it->kb[x], from);
        it->ke[x] = min(it->ke[x], to);
        if (it->ke[x] <= it->kb[x]) it->kb[x] = it->ke[x] = 0;
      }
      it->ub = from;
      it->ue = to;
    }
  }
  return true;
}

// The polynomial of fa::CapParams without its leading factor s, of u = s^2.
__device__ __forceinline__ uint64_t cap_poly(const fa::CapParams& c, uint64_t u) {
  uint64_t t = f2_fma(u, f2_pack(c.a[4], c.a[4]), f2_pack(c.a[3], c.a[3]));
  t = f2_fma(u, t, f2_pack(c.a[2], c.a[2]));
  t = f2_fma(u, t, f2_pack(c.a[1], c.a[1]));
  return f2_fma(u, t, f2_pack(c.a[0], c.a[0]));
}

// Bits of the columns [lo, lim).
__device__ __forceinline__ void interval_bits(int lo, int lim, uint32_t (&vis)[BN / 32]) {
#pragma unroll
  for (int k = 0; k < BN / 32; ++k) {
    const int from = min(max(lo - 32 * k, 0), 32), to = min(max(lim - 32 * k, 0), 32);
    vis[k] = (uint32_t)(((1ull << to) - 1) & ~((1ull << from) - 1));
  }
}

// Plans whose documents are not in order: takes the keys of other documents out
// of vis, unless every row of the warp has the document of the whole key tile
// (then false).
__device__ __noinline__ bool document_bits(uint32_t (&vis)[BN / 32], const ScoredFwdParams& p, int batch, int kv0,
                                           int my_doc) {
  const size_t tile = (size_t)batch * p.kv_tiles + kv0 / BN;
  const int lo = p.plan.tile_doc_lo[tile], hi = p.plan.tile_doc_hi[tile];
  if (__all_sync(0xffffffffu, lo == my_doc && hi == my_doc)) return false;
  const int* doc = p.plan.k_doc + tile * BN;
  for (int k = 0; k < BN / 32; ++k) {
    uint32_t bits = 0u;
    for (int c = 0; c < 32; ++c) bits |= (uint32_t)(__ldg(doc + 32 * k + c) == my_doc) << c;
    vis[k] &= bits;
  }
  return true;
}

// The distance bias of one row and key tile is a line in the column: it rises up to
// the row's own position and falls from there on (or all the way, where the tile
// starts there).  slope2: bias per step of the distance (log2 units); rel0: key of
// column 0 minus the row's position.
struct BiasLine {
  float s2, rel;     // per column; rel0
  uint64_t step[4];  // s2 * (0, 1), (2, 3), (4, 5), (6, 7)
  __device__ __forceinline__ BiasLine(int rel0, float slope2) : s2(rel0 >= 0 ? -slope2 : slope2), rel((float)rel0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) step[k] = f2_pack((float)(2 * k) * s2, (float)(2 * k + 1) * s2);
  }
  // Bias of column g (a multiple of 8) plus `more`.  rel + g is exact: a key near
  // the row is biased by few steps, so nothing large cancels there.
  __device__ __forceinline__ float at(int g, float more) const { return fmaf(rel + (float)g, s2, more); }
};

__device__ __forceinline__ uint64_t pair_of(const uint32_t (&s)[32], int c) {
  return f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
}

// One key tile of a capped row whose cap bounds every score (kBounded).  P = 2^x,
// with slopes 2^(x + bias - m_ref), needs no running maximum: m_ref is the
// greatest bias of a key the row sees.  So the scores stream through 32 or 64 columns
// at a time, each written back as bf16 P over scores already read.  The cap is
// taken by its polynomial; from the first score beyond it on (in any row of the
// warp), the rest of the tile goes by the form that holds everywhere (the scores
// are still in TMEM).  Returns the row's sum of P, for L, and the sum that its O is
// divided by.
// MASKED: only the columns in vis4 count, and the row's position may be inside
// the tile with visible keys on both sides.  Here the second sum is of P as rounded
// to bf16, so that a row of few keys is divided by the weights that its O was made
// of (with one key O is V exactly, as where a maximum makes its P 1).  In other
// tiles the roundings of 128 keys and more even out, and the two sums are one.
// Steps of 64 columns suit slopes (T 8192, d 128: 1090 -> 1060 us; T 2048, d 64: 89.6 ->
// 84.8) and not the cap alone (968 -> 1052).
// The loop stays rolled: unrolled, its instructions crowd the MMA thread's out of
// the instruction cache (T 8192, d 128: 964 us rolled, 997 unrolled; scores past the
// polynomial 1249 and 1403; T 2048, d 64: 82 and 96).  Two warpgroups of 64 columns
// each per tile were slower too (with the polynomial of degree 7, 925 us for one, 980
// to 1025 for two).
template <bool SLOPES, bool MASKED>
__device__ __forceinline__ float2 bounded_tile(uint32_t tS, const ScoredFwdParams& p, const uint32_t (&vis4)[BN / 32],
                                               int rel0, float slope2, float m_ref) {
  uint64_t rs[2] = {0ull, 0ull}, rounded = 0ull;
  bool small = true;
  BiasLine line(rel0, slope2);
  constexpr int W = SLOPES && !MASKED ? 64 : 32;  // columns at a time
#pragma unroll 1
  for (int ch = 0; ch < BN / W; ++ch) {
    const uint32_t vis = MASKED ? (ch < 2 ? (ch == 0 ? vis4[0] : vis4[1]) : (ch == 2 ? vis4[2] : vis4[3])) : 0u;
    const float relc = line.rel + (float)(W * ch);
    uint32_t s[W], pk[W / 2];
    auto load = [&]() {
#pragma unroll
      for (int w = 0; w < W; w += 32) tmem_ld32(tS + ch * W + w, *reinterpret_cast<uint32_t(*)[32]>(&s[w]));
      tmem_wait_ld();
    };
    auto two = [&](int c) { return f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])); };
    uint64_t part[2] = {0ull, 0ull};
    auto take = [&](int c, uint64_t x01, uint64_t x23) {  // four capped scores -> P and the sums
      float v0 = ex2(f2_lo(x01)), v1 = ex2(f2_hi(x01)), v2 = ex2(f2_lo(x23)), v3 = ex2(f2_hi(x23));
      if (MASKED) {
        if (!((vis >> c) & 1u)) v0 = 0.f;
        if (!((vis >> (c + 1)) & 1u)) v1 = 0.f;
        if (!((vis >> (c + 2)) & 1u)) v2 = 0.f;
        if (!((vis >> (c + 3)) & 1u)) v3 = 0.f;
      }
      part[0] = f2_add(part[0], f2_pack(v0, v1));
      part[1] = f2_add(part[1], f2_pack(v2, v3));
      pk[c / 2] = pack_bf16x2(v0, v1);
      pk[c / 2 + 1] = pack_bf16x2(v2, v3);
    };
    // the bias of columns c, c + 1 of this chunk plus `more`
    auto bias = [&](int c, float more) -> uint64_t {
      if (!SLOPES) return f2_pack(more, more);
      if (MASKED) {
        const float far0 = fabsf(relc + (float)c), far1 = fabsf(relc + (float)(c + 1));
        return f2_pack(fmaf(far0, -slope2, more - m_ref), fmaf(far1, -slope2, more - m_ref));
      }
      const float g = fmaf(relc + (float)(c & ~7), line.s2, more - m_ref);
      return f2_add(line.step[(c & 7) / 2], f2_pack(g, g));
    };
    if (small) {
      load();
      float top = 0.f;  // greatest s^2
#pragma unroll
      for (int c = 0; c < W; c += 4) {
        const uint64_t u01 = f2_mul(two(c), two(c)), u23 = f2_mul(two(c + 2), two(c + 2));
        top = fmax3(fmax3(top, f2_lo(u01), f2_hi(u01)), f2_lo(u23), f2_hi(u23));
        const uint64_t t01 = cap_poly(p.cap, u01), t23 = cap_poly(p.cap, u23);
        if (SLOPES)
          take(c, f2_fma(two(c), t01, bias(c, 0.f)), f2_fma(two(c + 2), t23, bias(c + 2, 0.f)));
        else
          take(c, f2_mul(two(c), t01), f2_mul(two(c + 2), t23));
      }
      small = !__any_sync(0xffffffffu, top > p.cap.small2);
    }
    if (!small) {
      const uint64_t in2 = f2_pack(p.cap.in, p.cap.in), m2cap2 = f2_pack(-2.f * p.cap.log2c, -2.f * p.cap.log2c);
      part[0] = part[1] = 0ull;
      load();
#pragma unroll
      for (int c = 0; c < W; c += 4) {
        uint64_t r01, r23, e01, e23;
        cap_quad<true>(f2_mul(two(c), in2), f2_mul(two(c + 2), in2), r01, r23, e01, e23);
        take(c, f2_fma(r01, m2cap2, bias(c, p.cap.log2c)), f2_fma(r23, m2cap2, bias(c + 2, p.cap.log2c)));
      }
    }
    rs[0] = f2_add(rs[0], part[0]);
    rs[1] = f2_add(rs[1], part[1]);
    if (MASKED) {
#pragma unroll
      for (int c = 0; c < W / 2; ++c)
        rounded = f2_add(rounded, f2_pack(__uint_as_float(pk[c] << 16), __uint_as_float(pk[c] & 0xffff0000u)));
    }
#pragma unroll
    for (int w = 0; w < W / 2; w += 16) tmem_st16(tS + W / 2 * ch + w, *reinterpret_cast<uint32_t(*)[16]>(&pk[w]));
  }
  const uint64_t rs2 = f2_add(rs[0], rs[1]);
  const float sum = f2_lo(rs2) + f2_hi(rs2);
  return make_float2(sum, MASKED ? f2_lo(rounded) + f2_hi(rounded) : sum);
}

// Slopes without a cap: two passes over the scores in TMEM.  Held in registers from one
// pass to the other they save nothing (T 8192, d 128: 959 us both ways; T 2048, d 64: 75.3
// against 74.4), and the masked tiles' passes, 32 columns at a time, stay short (see
// bounded_tile on code).
//
// First pass: the greatest score with its bias in one row and key tile (log2 units),
// or a little more: of eight columns, the greatest score with the greatest bias,
// which is over by at most seven steps of the slope.  Any reference near the
// maximum serves the softmax.  MASKED: every visible column by itself (also where
// seven steps of the slope are many).
template <bool MASKED>
__device__ __forceinline__ float line_max(uint32_t tS, float scale, const uint32_t (&vis4)[BN / 32], int rel0,
                                          float slope2) {
  float top[2] = {-__int_as_float(0x7f800000), -__int_as_float(0x7f800000)};
  const BiasLine line(rel0, slope2);
  if (MASKED) {
#pragma unroll 1
    for (int ch = 0; ch < BN / 32; ++ch) {
      const uint32_t vis = ch < 2 ? (ch == 0 ? vis4[0] : vis4[1]) : (ch == 2 ? vis4[2] : vis4[3]);
      const float relc = line.rel + (float)(32 * ch);
      uint32_t s[32];
      tmem_ld32(tS + ch * 32, s);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float x = fmaf(__uint_as_float(s[c]), scale, -slope2 * fabsf(relc + (float)c));
        if ((vis >> c) & 1u) top[c & 1] = fmaxf(top[c & 1], x);
      }
    }
  } else {
    uint32_t s[BN];
#pragma unroll
    for (int ch = 0; ch < BN / 32; ++ch) tmem_ld32(tS + ch * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[ch * 32]));
    tmem_wait_ld();
    const float more = fmaxf(0.f, 7.f * line.s2);
#pragma unroll
    for (int g = 0; g < BN; g += 8) {
      auto f = [&](int c) { return __uint_as_float(s[g + c]); };
      const float m = fmax3(fmax3(f(0), f(1), f(2)), fmax3(f(3), f(4), f(5)), fmaxf(f(6), f(7)));
      top[(g >> 3) & 1] = fmaxf(top[(g >> 3) & 1], fmaf(m, scale, line.at(g, more)));
    }
  }
  return fmaxf(top[0], top[1]);
}
// Second pass: P = 2^(score + bias - base) as bf16 over the scores; returns the row's
// sum of P.  Whole tiles take all columns at once, so that one wait for TMEM serves
// them (32 / 64 / 128 columns: T 8192 991, 967, 960 us; T 2048, d 64 75.6, 75.9, 74.4).
template <bool MASKED>
__device__ __forceinline__ float line_exp(uint32_t tS, float scale, const uint32_t (&vis4)[BN / 32], int rel0,
                                          float slope2, float base) {
  uint64_t rs[2] = {0ull, 0ull};
  const BiasLine line(rel0, slope2);
  const uint64_t scale2 = f2_pack(scale, scale);
  constexpr int W = MASKED ? 32 : BN;  // columns at a time
#pragma unroll 1
  for (int ch = 0; ch < BN / W; ++ch) {
    const uint32_t vis = MASKED ? (ch < 2 ? (ch == 0 ? vis4[0] : vis4[1]) : (ch == 2 ? vis4[2] : vis4[3])) : 0u;
    const float relc = line.rel + (float)(W * ch);
    uint32_t s[W];
#pragma unroll
    for (int w = 0; w < W / 32; ++w) tmem_ld32(tS + ch * W + w * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[w * 32]));
    tmem_wait_ld();
#pragma unroll
    for (int w = 0; w < W; w += 32) {
      uint32_t pk[16];
#pragma unroll
      for (int c = w; c < w + 32; c += 2) {
        uint64_t bias;
        if (MASKED) {
          bias = f2_pack(fmaf(fabsf(relc + (float)c), -slope2, -base), fmaf(fabsf(relc + (float)(c + 1)), -slope2, -base));
        } else {
          const float g = fmaf(relc + (float)(c & ~7), line.s2, -base);
          bias = f2_add(line.step[(c & 7) / 2], f2_pack(g, g));
        }
        const uint64_t x = f2_fma(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, bias);
        float v0 = ex2(f2_lo(x)), v1 = ex2(f2_hi(x));
        if (MASKED) {
          if (!((vis >> c) & 1u)) v0 = 0.f;
          if (!((vis >> (c + 1)) & 1u)) v1 = 0.f;
        }
        rs[(c >> 1) & 1] = f2_add(rs[(c >> 1) & 1], f2_pack(v0, v1));
        pk[(c - w) / 2] = pack_bf16x2(v0, v1);
      }
      tmem_st16(tS + (W * ch + w) / 2, pk);
    }
  }
  const uint64_t rs2 = f2_add(rs[0], rs[1]);
  return f2_lo(rs2) + f2_hi(rs2);
}

// Adds per_step * (key - position) to the scores of keys past the row's position.
__device__ __forceinline__ void turn_over(uint32_t (&sr)[BN], int rel0, float per_step) {
#pragma unroll
  for (int c = 0; c < BN; ++c)
    if (rel0 + c > 0 && rel0 < 0)
      sr[c] = __float_as_uint(fmaf((float)(rel0 + c), per_step, __uint_as_float(sr[c])));
}

// Capped scores of one row and key tile, in place: raw q.k -> log2 units with the
// cap and the distance bias (caps too wide for the bounded form, and slopes with plans
// that compare documents key by key).  The form that holds everywhere serves all
// scores, off by at most 2^-20 of the cap (L: 2e-4 under a cap of 1000), where the
// backward takes the polynomial on small ones: by 32 columns at a time here it cost
// 1309 -> 1387 us (T 8192, d 128, cap 100), and 1385 -> 1753 where scores pass it.  crossing: keys on both sides of the row's
// position may be visible; the rising line is then turned over past it.  (Two
// forms of the whole, each in a branch of its own, cost a move per score where
// the branches meet: 1870 against 2550 cycles a tile with slopes alone.)
template <bool SLOPES>
__device__ __forceinline__ void cap_scores(uint32_t (&sr)[BN], const ScoredFwdParams& p, int rel0, float slope2,
                                           bool crossing) {
  const uint64_t in2 = f2_pack(p.cap.in, p.cap.in), cap2 = f2_pack(p.cap.log2c, p.cap.log2c);
  const uint64_t m2cap2 = f2_pack(-2.f * p.cap.log2c, -2.f * p.cap.log2c);
  const BiasLine line(rel0, slope2);
#pragma unroll
  for (int c = 0; c < BN; c += 4) {
    const uint64_t s01 = f2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
    const uint64_t s23 = f2_pack(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
    uint64_t r01, r23, e01, e23, b01 = cap2, b23 = cap2;
    cap_quad<true>(f2_mul(s01, in2), f2_mul(s23, in2), r01, r23, e01, e23);
    if (SLOPES) {
      const float g = line.at(c & ~7, p.cap.log2c);
      b01 = f2_add(line.step[(c & 7) / 2], f2_pack(g, g));
      b23 = f2_add(line.step[(c & 7) / 2 + 1], f2_pack(g, g));
    }
    const uint64_t x01 = f2_fma(r01, m2cap2, b01), x23 = f2_fma(r23, m2cap2, b23);
    sr[c] = __float_as_uint(f2_lo(x01));
    sr[c + 1] = __float_as_uint(f2_hi(x01));
    sr[c + 2] = __float_as_uint(f2_lo(x23));
    sr[c + 3] = __float_as_uint(f2_hi(x23));
  }
  if (SLOPES && crossing) turn_over(sr, rel0, -2.f * slope2);
}

// Plans whose documents are not in order: hides the keys of other documents one
// by one, unless every row of the warp has the document of the whole key tile.
__device__ __forceinline__ void mask_documents(uint32_t (&sr)[BN], const ScoredFwdParams& p, int batch, int kv0, int my_doc) {
  const size_t tile = (size_t)batch * p.kv_tiles + kv0 / BN;
  const int lo = p.plan.tile_doc_lo[tile], hi = p.plan.tile_doc_hi[tile];
  if (__all_sync(0xffffffffu, lo == my_doc && hi == my_doc)) return;
  const int4* doc = reinterpret_cast<const int4*>(p.plan.k_doc + tile * BN);
  const uint32_t hidden = 0xff800000u;  // -inf
#pragma unroll
  for (int c = 0; c < BN; c += 4) {
    const int4 dk = __ldg(doc + c / 4);
    if (dk.x != my_doc) sr[c] = hidden;
    if (dk.y != my_doc) sr[c + 1] = hidden;
    if (dk.z != my_doc) sr[c + 2] = hidden;
    if (dk.w != my_doc) sr[c + 3] = hidden;
  }
}

// WINDOW (causal only): the sliding-window terms are compiled in only where
// a window is set, so the plain causal and full masks keep their lean code.
// SCORE: kPlain, or the score-modified form (CAUSAL and WINDOW are then not used).
template <int HD, int HDV, bool CAUSAL, bool WINDOW, int SCORE>
__global__ void __launch_bounds__(kThreads, 1)
    fa_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const FwdParamsOf<SCORE> p) {
  using C = FwdCfg<HD, HDV>;
  constexpr int NS = C::NS;
  if constexpr (SCORE >= 0) grid_next();
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars;           // [2] per tile
  uint64_t* q_empty = q_full + 2;    // [2]
  // One "full" barrier per ring slot covers both K_j and V_j, so the MMA
  // thread checks a key tile once; K and V are released separately (K after
  // the last S that reads it, V after the last P.V), so K_{j+NS} can load
  // before V_j's readers are done.
  uint64_t* kv_full = q_empty + 2;
  uint64_t* k_empty = kv_full + NS;
  uint64_t* v_empty = k_empty + NS;
  uint64_t* s_full = v_empty + NS;  // [2] per tile
  uint64_t* p_full = s_full + 2;    // [2]
  uint64_t* o_done = p_full + 2;    // [2]
  uint64_t* drain = o_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t q_buf = smem_u32(smem + C::OFF_Q);
  const uint32_t k_base = smem_u32(smem + C::OFF_K);
  const uint32_t v_base = smem_u32(smem + C::OFF_V);
  bool withhold_q = false;
#ifdef FA_TEST_HOOKS
  withhold_q = p.test_withhold_q != 0;
#endif

  // Producer state; the first item's Q and its first NS key/value tiles (the
  // ring slots are all free) are issued during set-up, before TMEM allocation
  // and the CTA-wide barrier, so their memory latency overlaps the set-up.
  int nq[2] = {0, 0};  // Q_X loads issued (the producer) / waited for (the MMA thread)
  int pre_kv = 0;      // key/value tiles of item 0 issued during set-up
  auto load_q = [&](const FwdItem& it, int x) {
    if (!withhold_q) {
      mbar_arrive_expect_tx(&q_full[x], C::Q_BYTES);
#pragma unroll
      for (int cb = 0; cb < HD / 64; ++cb)
        tma_load_3d(smem + C::OFF_Q + x * C::Q_BYTES + cb * BM * 128, &tmQ, &q_full[x], cb * 64, it.q0 + x * BM,
                    it.bh);
    }
    ++nq[x];
  };
  auto load_k = [&](const FwdItem& it, int jj, int s) {
    mbar_arrive_expect_tx(&kv_full[s], C::K_BYTES + C::V_BYTES);
#pragma unroll
    for (int cb = 0; cb < HD / 64; ++cb)
      tma_load_3d(smem + C::OFF_K + s * C::K_BYTES + cb * BN * 128, &tmK, &kv_full[s], cb * 64,
                  (it.ub + jj) * BN, it.bkv);
  };
  auto load_v = [&](const FwdItem& it, int jj, int s) {
#pragma unroll
    for (int cb = 0; cb < HDV / 64; ++cb)
      tma_load_3d(smem + C::OFF_V + s * C::V_BYTES + cb * BN * 128, &tmV, &kv_full[s], cb * 64,
                  (it.ub + jj) * BN, it.bkv);
  };

  if (threadIdx.x == 0) {
    *abort_flag = (smem_u32(smem) & 1023u) ? 1 : 0;  // swizzled tiles need 1024 B alignment
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 128);
      mbar_init(&o_done[x], 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    FwdItem it;
    if (*abort_flag == 0 && fwd_item<CAUSAL, WINDOW, SCORE>(p, 0, &it)) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (it.ke[x] > it.kb[x]) load_q(it, x);
      for (; pre_kv < NS && pre_kv < it.ue - it.ub; ++pre_kv) {
        load_k(it, pre_kv, pre_kv);
        load_v(it, pre_kv, pre_kv);
      }
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool run = *abort_flag == 0;

  if (warp < 4) {
    setmaxnreg_dec<kRegsLow>();
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0 && run) {
        int g = pre_kv;     // ring position of the next key/value tile (running over items)
        int kv_last[NS];    // last ring pass whose K and V loads were both issued, per slot
        bool half = false;  // a K load was issued whose V load was not (abort in between)
#pragma unroll
        for (int s = 0; s < NS; ++s) kv_last[s] = s < pre_kv ? 0 : -1;
        bool ok = true;
        FwdItem it;
        for (int n = 0; ok && fwd_item<CAUSAL, WINDOW, SCORE>(p, n, &it); ++n) {
          if (n > 0) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (it.ke[x] <= it.kb[x]) continue;
              // Q_X's buffer is free once the previous item's last S_X has read it.
              if (nq[x] > 0 && !fwd_wait(&q_empty[x], (nq[x] - 1) & 1, abort_flag)) { ok = false; break; }
              load_q(it, x);
            }
          }
          for (int jj = n == 0 ? pre_kv : 0; ok && jj < it.ue - it.ub; ++jj, ++g) {
            const int s = g % NS, u = g / NS;
            if (!fwd_wait(&k_empty[s], (u & 1) ^ 1, abort_flag)) { ok = false; break; }
            load_k(it, jj, s);
            half = true;
            if (!fwd_wait(&v_empty[s], (u & 1) ^ 1, abort_flag)) { ok = false; break; }
            load_v(it, jj, s);
            half = false;
            kv_last[s] = u;
          }
        }
        // Every issued copy must land before the CTA releases its shared memory.
        if (!withhold_q)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (nq[x] > 0) mbar_wait_bounded(&q_full[x], (nq[x] - 1) & 1);
#pragma unroll
        for (int s = 0; s < NS; ++s)
          if (kv_last[s] >= 0) mbar_wait_bounded(&kv_full[s], kv_last[s] & 1);
        // A K load whose V never followed leaves its barrier short of bytes:
        // give the copy in flight time to land before the CTA exits.
        if (half) {
          const uint64_t t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 1000000ull) {
          }
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0 && run) {
        constexpr uint32_t idS = idesc_bf16(BM, BN, 0, 0);
        constexpr uint32_t idPV = idesc_bf16(BM, HDV, 0, 1);
        int np[2] = {0, 0};  // p_full phases waited for, per tile
        int base = 0;        // ring position of the current item's first key tile
        bool ok = true;
        FwdItem it;
        for (int n = 0; ok && fwd_item<CAUSAL, WINDOW, SCORE>(p, n, &it); ++n) {
          auto active = [&](int x, int j) { return j >= it.kb[x] && j < it.ke[x]; };
          // S_X(j) = Q_X K_j^T into TMEM [128 X, 128 X + 128).  Every barrier
          // check here costs the tensor pipe a shared-memory round trip, so
          // K_j / V_j are checked only where nothing else vouches for them
          // (wait_kv): tile B's S uses the key tile tile A has just waited
          // for, and with KV_VIA_SOFTMAX, inside an item, the P_X(j-1)
          // barrier waited for just before covers them too (the softmax
          // checks K_j / V_j before it arrives).
          auto issue_s = [&](int x, int j, bool wait_kv) -> bool {
            const int pos = base + (j - it.ub), s = pos % NS;
            if (j == it.kb[x]) {  // the tile's first S of this item: wait for its Q
              if (!fwd_wait(&q_full[x], nq[x] & 1, abort_flag)) return false;
              ++nq[x];
            }
            if (wait_kv && !fwd_wait(&kv_full[s], (pos / NS) & 1, abort_flag)) return false;
            tc_fence_after();
            const uint64_t a0 = desc_kmajor(q_buf + x * C::Q_BYTES), b0 = desc_kmajor(k_base + s * C::K_BYTES);
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
              const uint32_t step = (k >> 2) * (BM * 128) + (k & 3) * 32;
              mma_ss(tmem + x * 128, desc_at(a0, step), desc_at(b0, step), idS, k > 0 ? 1u : 0u);
            }
            mma_commit(&s_full[x]);
            if (j == it.ke[x] - 1) mma_commit(&q_empty[x]);  // last reader of Q_X in this item
            return true;
          };
          // O_X += P_X(j) V_j with P_X read from TMEM (packed bf16 over S_X)
          auto issue_pv = [&](int x, int j) -> bool {
            const int s = (base + j - it.ub) % NS;
            // V_j landed with K_j: the S(j) MMA before this P.V waited for both.
            if (!fwd_wait(&p_full[x], np[x] & 1, abort_flag)) return false;
            ++np[x];
            tc_fence_after();
            const uint64_t v0 = desc_mnmajor(v_base + s * C::V_BYTES, BN * 128);
#pragma unroll
            for (int k = 0; k < BN / 16; ++k) {
              const uint64_t bd = desc_at(v0, k * 2048);
              mma_ts(tmem + 256 + x * 128, tmem + x * 128 + k * 8, bd, idPV, (j > it.kb[x] || k > 0) ? 1u : 0u);
            }
            return true;
          };
          if (it.ue > it.ub) {
            // A tile whose range starts at ub gets its first S up front; tile B,
            // if it starts later, gets it in the loop below one step before its range.
            if (ok && active(0, it.ub)) ok = issue_s(0, it.ub, true);
            if (ok && active(1, it.ub)) ok = issue_s(1, it.ub, !active(0, it.ub));
            if (ok) mma_commit(&k_empty[base % NS]);
          }
          for (int j = it.ub; ok && j < it.ue; ++j) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (active(x, j)) {
                if (!issue_pv(x, j)) { ok = false; break; }
                if (x == 1 || !active(1, j)) mma_commit(&v_empty[(base + j - it.ub) % NS]);  // last reader of V_j
              }
              if (active(x, j + 1)) {
                // Tile B relies on tile A's wait (or, with KV_VIA_SOFTMAX, on
                // A's P_A(j) when A goes on to j + 1); with KV_VIA_SOFTMAX a
                // tile's own P_X(j), just waited for, vouches for K_{j+1} / V_{j+1}.
                const bool covered = (x == 1 && active(0, j + 1) && (!C::KV_VIA_SOFTMAX || active(0, j))) ||
                                     (C::KV_VIA_SOFTMAX && active(x, j));
                if (!issue_s(x, j + 1, !covered)) { ok = false; break; }
                if (x == 1 || !active(1, j + 1))
                  mma_commit(&k_empty[(base + j + 1 - it.ub) % NS]);  // last reader of K_{j+1}
              } else if (active(x, j)) {
                mma_commit(&o_done[x]);
              }
            }
          }
          base += it.ue - it.ub;
        }
        // Let every MMA issued above finish before TMEM is released.
        mma_commit(drain);
        mbar_wait_bounded(drain, 0);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue of tile x
    setmaxnreg_inc<kRegsHigh>();
    const int x = (warp - 4) >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;  // row inside the tile == TMEM lane
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_base;
    const uint32_t tO = tmem + 256 + x * 128 + lane_base;
    constexpr bool CAP = SCORE >= 0 && (SCORE & fa::kCap), SLOPES = SCORE >= 0 && (SCORE & fa::kSlopes);
    constexpr bool BOUNDED = SCORE >= 0 && (SCORE & fa::kBounded);
    const float sl2 = CAP ? 1.f : p.scale_log2;  // what brings the (capped) scores to log2 units
    const float NEG_INF = -__int_as_float(0x7f800000);
    int ns = 0, no = 0;  // s_full / o_done phases waited for
    int base = 0;        // ring position of the current item's first key tile
    bool ok = run;
    // What a row's mask and bias need (SCORE >= 0), read from the plan or worked out.
    struct Row {
      int lo = 0, hi = 0;  // the keys it sees
      int doc = 0;         // its document, where the plan wants documents compared key by key
      int pos = 0, batch = 0;  // its position among Tq, its batch entry
      bool by_key = false;
      float slope2 = 0.f;  // bias per step of the distance, log2 units
    };
    auto row_of = [&](const FwdItem& it) -> Row {
      Row w;
      if constexpr (SCORE >= 0) {
        const int i = it.q0 + x * BM + r;
        w.pos = i;
        w.batch = it.bh / p.Hq;
        // (packed heads: the row's position, and its head, within the group)
        int head = 0;
        if (kIsFew<SCORE> && p.row_mod) {
          const int row = min(i, p.Tq - 1);
          head = row / p.row_mod;
          w.pos = row - head * p.row_mod;
        }
        if (p.plan.kv_beg) {
          const size_t at = (size_t)w.batch * p.q_tiles * BM + (i < p.Tq ? w.pos : 0);
          w.lo = p.plan.row_lo[at];
          w.hi = i < p.Tq ? min(p.plan.row_hi[at], p.Tk) : 0;
          w.doc = p.plan.q_doc[at];
          w.by_key = fa::plan_flag(p.plan.by_key, w.batch);
        } else {
          w.lo = max(0, w.pos + p.lo_off);
          w.hi = min(p.Tk, w.pos + p.hi_off);
        }
        if (SLOPES)
          w.slope2 = p.slopes[(it.bh - w.batch * p.Hq) * (kIsFew<SCORE> ? p.group : 1) + head] * 1.4426950408889634f;
      }
      return w;
    };
    FwdItem it, next;
    bool more = fwd_item<CAUSAL, WINDOW, SCORE>(p, 0, &it);
    Row row, next_row;
    if (more) row = row_of(it);
    for (int n = 0; ok && more; ++n, it = next, row = next_row) {
      const int item_base = base;
      base += it.ue - it.ub;
      const int kbx = x ? it.kb[1] : it.kb[0];  // first key tile of this tile's range
      const int nkv = (x ? it.ke[1] : it.ke[0]) - kbx;
      const int qx0 = it.q0 + x * BM;
      const int i = qx0 + r;  // query row
      const int row_lo = row.lo, row_hi = row.hi, my_doc = row.doc, pos = row.pos, batch = row.batch;
      const bool by_key = row.by_key;
      const float slope2 = row.slope2;
      // reference max (log2 units) the P values are taken against
      float m_ref = NEG_INF;
      if (BOUNDED && !(SLOPES && by_key)) {
        m_ref = 0.f;
        if (SLOPES) {  // the greatest bias: of the nearest key the row sees, or the farthest (negative slopes)
          const int to_lo = pos + p.causal_off - row_lo, to_hi = pos + p.causal_off - (row_hi - 1);
          const int near = to_lo >= 0 && to_hi <= 0 ? 0 : min(abs(to_lo), abs(to_hi));
          m_ref = -slope2 * (float)(slope2 >= 0.f ? near : max(abs(to_lo), abs(to_hi)));
        }
      }
      float l = 0.f, l_o = 0.f;  // sum of P; (BOUNDED) the sum that O is divided by
      for (int jx = 0; ok && jx < nkv; ++jx) {  // jx-th key tile of this tile's range
        // the warp agrees on the outcome before its collective TMEM loads
        if (!__all_sync(0xffffffffu, fwd_wait(&s_full[x], ns & 1, abort_flag))) { ok = false; break; }
        ++ns;
        tc_fence_after();
        const int kv0 = (kbx + jx) * BN;
        int lim = 0, lo = 0, rel0 = 0;  // (SCORE >= 0) columns [lo, lim) are visible to row i; column 0 minus its position
        bool crossing = false;          // some row of the warp may see keys on both sides of its position in this tile
        if constexpr (SCORE >= 0) {
          lim = row_hi - kv0;
          lo = row_lo - kv0;
          rel0 = kv0 - p.causal_off - pos;
          if (SLOPES) crossing = p.two_sided && __any_sync(0xffffffffu, rel0 < 0 && rel0 + BN > 1);
        }
        if (BOUNDED && !(SLOPES && by_key)) {
          if constexpr (BOUNDED) {
            uint32_t vis[BN / 32];
            bool masked = crossing || __any_sync(0xffffffffu, lim < BN || lo > 0);
            if (masked || by_key) {
              interval_bits(lo, lim, vis);
              if (by_key) masked = document_bits(vis, p, batch, kv0, my_doc) || masked;
            }
            const float2 sums = masked ? bounded_tile<SLOPES, true>(tS, p, vis, rel0, slope2, m_ref)
                                       : bounded_tile<SLOPES, false>(tS, p, vis, rel0, slope2, m_ref);
            l += sums.x;
            l_o += sums.y;
          }
        } else {
          constexpr bool LINE = SLOPES && !CAP;  // two passes over the scores in TMEM
          uint32_t sr[BN], vis[BN / 32];         // the scores (in registers), or which columns count (LINE)
          bool masked = false;
          float mt2;  // row max, in log2 units
          if constexpr (LINE) {
            // (the warp takes one way: the ways load TMEM, and packed rows' slopes differ)
            const bool steep = __any_sync(0xffffffffu, fabsf(slope2) > 8.f);
            masked = crossing || __any_sync(0xffffffffu, lim < BN || lo > 0);
            if (masked || by_key || steep) {
              interval_bits(lo, lim, vis);
              if (by_key) masked = document_bits(vis, p, batch, kv0, my_doc) || masked;
              masked = masked || steep;
            }
            mt2 = masked ? line_max<true>(tS, sl2, vis, rel0, slope2) : line_max<false>(tS, sl2, vis, rel0, slope2);
          } else {
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
            tmem_wait_ld();
            if constexpr (SCORE >= 0) {
              if constexpr (CAP) cap_scores<SLOPES>(sr, p, rel0, slope2, crossing);
              // (one end at a time: a tile seldom has both, and a loop over both is half
              // as long again; packed documents 154 -> 141 us)
              if (__any_sync(0xffffffffu, lim < BN)) {
#pragma unroll
                for (int c = 0; c < BN; ++c)
                  if (c >= lim) sr[c] = __float_as_uint(NEG_INF);
              }
              if (__any_sync(0xffffffffu, lo > 0)) {
#pragma unroll
                for (int c = 0; c < BN; ++c)
                  if (c < lo) sr[c] = __float_as_uint(NEG_INF);
              }
              if (by_key) mask_documents(sr, p, batch, kv0, my_doc);
            } else {
              // window: the tile's last row starts its window past this key tile's start
              const bool win_mask = WINDOW && qx0 + BM - 1 + p.causal_off - p.window + 1 > kv0;
              const bool need_mask = (kv0 + BN > p.Tk) || (CAUSAL && kv0 + BN - 1 > qx0 + p.causal_off) || win_mask;
              if (need_mask) {
                int lim = p.Tk - kv0;  // columns [lo, lim) are visible to row i
                if (CAUSAL) lim = min(lim, i + p.causal_off + 1 - kv0);
                const int lo = win_mask ? i + p.causal_off - p.window + 1 - kv0 : -BN;
#pragma unroll
                for (int c = 0; c < BN; ++c)
                  if (c >= lim || c < lo) sr[c] = __float_as_uint(NEG_INF);
              }
            }
            // row max: eight independent three-input max chains (short dependency depth)
            float pm[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) pm[k] = __uint_as_float(sr[k]);
#pragma unroll
            for (int c = 8; c + 16 <= BN; c += 16)
#pragma unroll
              for (int k = 0; k < 8; ++k) pm[k] = fmax3(pm[k], __uint_as_float(sr[c + k]), __uint_as_float(sr[c + 8 + k]));
#pragma unroll
            for (int k = 0; k < 8; ++k) pm[k] = fmaxf(pm[k], __uint_as_float(sr[BN - 8 + k]));
            const float mt = fmax3(fmax3(pm[0], pm[1], pm[2]), fmax3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7]));
            mt2 = mt * sl2;
          }
          float m_new = m_ref;
          if (mt2 > m_ref + kRescaleThreshold) m_new = mt2;  // also taken when m_ref == -inf
          // Does this row's O need rescaling, and does any row of the warp's?  (The
          // vote is taken here, where fewer registers are live than after exp2.)
          const bool rescale = jx > 0 && m_new != m_ref && m_ref != NEG_INF;
          const bool warp_rescale = __any_sync(0xffffffffu, rescale);
          const float base = (m_new == NEG_INF) ? 0.f : m_new;
          float rowsum;
          if constexpr (LINE) {
            rowsum = masked ? line_exp<true>(tS, sl2, vis, rel0, slope2, base)
                            : line_exp<false>(tS, sl2, vis, rel0, slope2, base);
          } else {
            const uint64_t sl2x2 = f2_pack(sl2, sl2), nbase2 = f2_pack(-base, -base);
            // exponentials (argument and row sum on packed pairs); P (packed bf16)
            // goes over the already-loaded scores in TMEM 16 columns at a time
            uint64_t rs[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint64_t xv = f2_fma(
                  f2_pack(__uint_as_float(sr[32 * c + 2 * e]), __uint_as_float(sr[32 * c + 2 * e + 1])), sl2x2, nbase2);
                const float e0 = ex2(f2_lo(xv)), e1 = ex2(f2_hi(xv));
                rs[e & 3] = f2_add(rs[e & 3], f2_pack(e0, e1));
                pk[e] = pack_bf16x2(e0, e1);
              }
              tmem_st16(tS + 16 * c, pk);
            }
            const uint64_t rs2 = f2_add(f2_add(rs[0], rs[1]), f2_add(rs[2], rs[3]));
            rowsum = f2_lo(rs2) + f2_hi(rs2);
          }
          // O_X is idle here: the P.V of tile j-1 completed before S_X(j) did.
          const float alpha = (m_new == m_ref) ? 1.f : (m_ref == NEG_INF ? 0.f : ex2(m_ref - m_new));
          l = l * alpha + rowsum;
          // TMEM loads and stores are warp-collective: when any row of the warp
          // must rescale its O row, every lane takes part (factor 1 where not).
          if (warp_rescale) {
            const float a = rescale ? alpha : 1.f;
#pragma unroll
            for (int c = 0; c < HDV / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
              tmem_st32(tO + c * 32, o);
            }
          }
          m_ref = m_new;
        }
        tmem_wait_st();
        tc_fence_before();
        // The MMA thread takes this barrier as word that K / V of this tile's
        // next key tile have landed too (it issues that S right after this
        // tile's P.V without checking them), so one thread checks them first.
        if (C::KV_VIA_SOFTMAX && r == 0 && jx + 1 < nkv) {
          const int pos = item_base + kbx + jx + 1 - it.ub;
          if (!fwd_wait(&kv_full[pos % NS], (pos / NS) & 1, abort_flag)) ok = false;
        }
        mbar_arrive(&p_full[x]);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      }
      // The next item is looked up here, where few registers are live and its loads
      // overlap the wait and the epilogue: the epilogue and the start of an item
      // are all that the MMA thread waits for between items.
      more = ok && fwd_item<CAUSAL, WINDOW, SCORE>(p, n + 1, &next);
      if (more) next_row = row_of(next);
      // ---- epilogue: O / l -> bf16 -> global (one row per thread); L -> global
      if (ok && nkv > 0) {
        if (!__all_sync(0xffffffffu, fwd_wait(&o_done[x], no & 1, abort_flag))) ok = false;
        ++no;
        tc_fence_after();
      }
      if (!BOUNDED || (SLOPES && by_key)) l_o = l;
      // (a tile past the last row, or tile B of a single-tile item, has nothing to write)
      if (!ok || qx0 >= p.Tq || (x == 1 && it.single)) continue;
      const bool row_ok = i < p.Tq;
      if constexpr (kIsFew<SCORE>) {
        if (p.split > 1) {  // the unnormalised row, its reference and sum, for fa_fwd_join
          const size_t row = ((size_t)fwd_index(n) * 2 + x) * BM + r;
          if (row_ok)
            reinterpret_cast<float4*>(p.part + (size_t)p.n_items * 2 * BM * HDV)[row] =
                make_float4(m_ref, nkv > 0 ? l : -1.f, l_o, 0.f);
          float4* out = reinterpret_cast<float4*>(p.part + row * HDV);
          if (nkv > 0) {
#pragma unroll
            for (int c = 0; c < HDV / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_wait_ld();
              if (row_ok) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  out[c * 8 + q] = make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                                               __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3]));
              }
            }
          }
          continue;
        }
      }
      // (l is 0 where the row saw no key, and NaN where one of its scores is: so are L and O then)
      if (row_ok) p.L[(size_t)it.bh * p.Tq + i] = l == 0.f ? NEG_INF : (m_ref + __log2f(l)) * 0.69314718055994531f;
      const float inv_l = l == 0.f ? 0.f : 1.f / l_o;
      uint4* orow = reinterpret_cast<uint4*>(p.O + ((size_t)it.bh * p.Tq + (row_ok ? i : 0)) * HDV);
#pragma unroll
      for (int c = 0; c < HDV / 32; ++c) {
        uint32_t o[32];
        if (nkv > 0) {
          tmem_ld32(tO + c * 32, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (row_ok) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(o[8 * q + 0]) * inv_l, __uint_as_float(o[8 * q + 1]) * inv_l);
            w.y = pack_bf16x2(__uint_as_float(o[8 * q + 2]) * inv_l, __uint_as_float(o[8 * q + 3]) * inv_l);
            w.z = pack_bf16x2(__uint_as_float(o[8 * q + 4]) * inv_l, __uint_as_float(o[8 * q + 5]) * inv_l);
            w.w = pack_bf16x2(__uint_as_float(o[8 * q + 6]) * inv_l, __uint_as_float(o[8 * q + 7]) * inv_l);
            orow[c * 4 + q] = w;
          }
        }
      }
    }
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
cudaError_t launch_fwd_t(const fa::Problem& pr, const fa::ScoreMods& mods, const fa::FwdShape& shape,
                         const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, void* O, float* L,
                         float* part, cudaStream_t stream) {
  using C = FwdCfg<HD, HDV>;
  const void* fn = reinterpret_cast<const void*>(fa_fwd_kernel<HD, HDV, CAUSAL, WINDOW, SCORE>);
  cudaError_t e = fa::allow_dynamic_smem(fn, C::SMEM);
  if (e != cudaSuccess) return e;
  // The register split only balances if every thread was launched with
  // exactly kRegsLaunch registers; otherwise the softmax warpgroups' request
  // could never be met, so refuse to launch.
  cudaFuncAttributes fa_attr;
  e = cudaFuncGetAttributes(&fa_attr, fn);
  if (e != cudaSuccess) return e;
  if (fa_attr.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
  const int sms = fa::sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  FwdParamsOf<SCORE> p;
  p.O = static_cast<uint16_t*>(O);
  p.L = L;
  p.status = fa::device_status_word();
  p.Hq = shape.heads;
  p.Hkv = pr.Hkv;
  p.G = shape.heads / pr.Hkv;
  p.Tq = shape.rows;
  p.Tk = pr.Tk;
  p.causal_off = pr.Tk - pr.Tq;
  p.window = pr.causal ? pr.window : 0;
  p.kv_tiles = pr.kv_tiles();
  p.n_bh = pr.B * shape.heads;
  p.n_pairs = (shape.rows + 2 * BM - 1) / (2 * BM);
  const long long n_pair_items = (long long)p.n_bh * p.n_pairs;
  // Without a causal mask every item has the same work.  A last round with at
  // most half as many items as SMs then runs them as single tiles on twice
  // as many SMs (a tile alone takes ~0.65 of a pair's time: no ping-pong).
  const long long r = n_pair_items % sms;
  p.n_full = (!pr.causal && !mods.plan && r > 0 && 2 * r <= sms) ? n_pair_items - r : n_pair_items;
  p.n_items = p.n_full + 2 * (n_pair_items - p.n_full);
  if (shape.split > 1) {
    p.n_full = n_pair_items;
    p.n_items = n_pair_items * shape.split;
  }
  p.scale_log2 = pr.scale * 1.4426950408889634f;
  if constexpr (SCORE >= 0) {
    p.cap = fa::cap_params(mods.softcap, pr.scale);
    p.slopes = mods.slopes;
    p.hi_off = fa::row_hi_off(pr);
    p.lo_off = fa::row_lo_off(pr);
    p.q_tiles = pr.q_tiles();
    p.two_sided = !pr.causal || mods.plan;
    p.row_mod = shape.row_mod;
    p.group = shape.group;
    p.split = shape.split;
    p.part = part;
    p.plan = fa::plan_view(pr, mods.plan);
  }
  p.test_withhold_q = fa::test_withhold() == fa::kWithholdFwdQ;
  const int grid = (int)(p.n_items < sms ? p.n_items : sms);
  fa_fwd_kernel<HD, HDV, CAUSAL, WINDOW, SCORE><<<grid, kThreads, C::SMEM, stream>>>(mq, mk, mv, p);
  return cudaGetLastError();
}

}  // namespace
