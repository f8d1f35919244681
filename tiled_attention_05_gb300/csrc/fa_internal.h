// Host-side glue shared by the forward, backward and API translation units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/fa.h"

namespace fa {

constexpr int kTile = 128;  // rows of a query tile and of a key/value tile

// Failure-path test hooks.  Only a separate test build of the library
// (compiled with FA_TEST_HOOKS) can make a producer withhold one load, so that
// a barrier is never completed and the kernel's bounded waits must expire;
// the product build has neither the switch nor the code behind it.
enum TestWithhold : int { kWithholdNone = 0, kWithholdFwdQ = 1, kWithholdBwdDO = 2 };
#ifdef FA_TEST_HOOKS
int test_withhold();
#else
constexpr int test_withhold() { return kWithholdNone; }
#endif

struct Problem {
  int B, Hq, Hkv, Tq, Tk, d, dv;  // d: Q/K head size, dv: V/O head size
  int causal;
  int window;   // causal sliding window in keys, 0 = none
  float scale;  // resolved (> 0)
  int G() const { return Hkv ? Hq / Hkv : 0; }  // (no heads at all are allowed)
  int q_tiles() const { return (Tq + kTile - 1) / kTile; }
  int kv_tiles() const { return (Tk + kTile - 1) / kTile; }
  long long Tq_pad() const { return (long long)q_tiles() * kTile; }
};

// Encodes a TMA descriptor for a contiguous bf16 tensor viewed as
// [outer][rows][inner] (inner contiguous), box = 64 x 128 x 1, 128-byte swizzle.
// Returns false if cuTensorMapEncodeTiled rejects it.
bool encode_rows_bf16(CUtensorMap* map, const void* base, int inner, int rows, long long outer);

// TMA descriptor for the fp32 dQ accumulator viewed as [outer][rows][inner]
// (inner = d), box = 32 x box_rows x 1 (128 bytes x box_rows), 128-byte swizzle.
bool encode_acc_f32(CUtensorMap* map, const void* base, int inner, long long rows, long long outer, int box_rows);

// Device status word of the current device (see fa_last_device_status).
int* device_status_word();

// Lets `kernel` use `bytes` of dynamic shared memory on the current device.
// The attribute is per device, so it is set once for each (kernel, device)
// pair; safe to call from several host threads.
cudaError_t allow_dynamic_smem(const void* kernel, int bytes);

// Launches one of the short kernels (mask plan, join, pre, cast, rotary) so that it may
// start while the one before it in the stream ends; it waits by itself (grid_previous)
// before it uses what others wrote.  Hot, and with inputs that change from call to
// call: a step of B 2, 16 heads of 128, T 2001, prefixes, 192 -> 186.4 us; rotary of
// 335 MB 55.4 -> 52.9.  The two large kernels only let the next one start: launched
// this way themselves, their CTAs reach the SMs in another order, and packed documents
// took 142 -> 153 us forward and 357 -> 394 backward.
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  c.attrs = attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// SM count of the current device; 0 if it cannot be read.
int sm_count();

// ---------------------------------------------------------------- score modifications
// Bits of the kernels' SCORE template argument; kPlain compiles none of it.
// kBounded (forward, with kCap): the cap keeps 2^score inside fp32, so the
// softmax needs no running maximum.
// kFew (forward): packed heads and split items (FwdShape).  (In every instance their
// bookkeeping cost the large calls 4%: T 8192, cap 50, with the polynomial of degree 7
// that was taken then, 938 -> 978 us.)
enum ScoreBits : int { kPlain = -1, kCap = 1, kSlopes = 2, kBounded = 4, kFew = 8 };

// Largest cap (log2 units) of the bounded form over Tk keys.  P is between 2^-90 and
// 2^90, a normal number of bf16 and fp32 (as are its products with values down to
// 2^-36), and a row's unnormalised O, at most 2^cap times the values' size times Tk,
// stays below 2^127 with values below 2^20: 2^90 up to 2^17 keys (in natural units a cap
// of 62), half as much for each further doubling.
constexpr int kBoundedCapLog2 = 90, kBoundedKeysLog2 = 127 - 20 - kBoundedCapLog2;
inline float bounded_cap_log2(int Tk) {
  int more = 0;
  while (((long long)Tk - 1) >> (kBoundedKeysLog2 + more) > 0) ++more;
  return (float)(kBoundedCapLog2 - more);
}

struct ScoreMods {
  float softcap = 0.f;            // c > 0: x = c tanh(x / c)
  const float* slopes = nullptr;  // [Hq]: x -= slope |i + Tk - Tq - j|
  const void* plan = nullptr;     // mask plan (documents, prefixes) for the same dims
  bool any() const { return softcap > 0.f || slopes || plan; }
  int bits() const { return (softcap > 0.f ? kCap : 0) | (slopes ? kSlopes : 0); }
  int fwd_bits(int Tk) const {
    return softcap > 0.f && softcap * 1.4426950408889634f <= bounded_cap_log2(Tk) ? bits() | kBounded : bits();
  }
};

// Without a plan, row i sees keys [i + lo_off, i + hi_off) within [0, Tk);
// kFar stands for "no limit" and keeps the sums inside 32 bits.
constexpr int kFar = 1 << 30;
inline int row_hi_off(const Problem& p) { return p.causal ? p.Tk - p.Tq + 1 : kFar; }
inline int row_lo_off(const Problem& p) { return p.causal && p.window ? p.Tk - p.Tq - p.window + 1 : -kFar; }

// The cap, for the kernels.  c * tanh(s * scale / c) in log2 units of a raw score s:
//   everywhere  log2c - 2 log2c / (1 + exp2(in * s));
//   for s^2 <= small2, i.e. arguments y = s * scale / c up to 1/2, where scores
//   mostly are (a cap of 50 and scores up to 25):  s * (a0 + u (a1 + ... + u a4)),
//   u = s^2.  The odd polynomial of degree 9 has the least greatest error there,
//   3.1e-9 of c (fitted to tanh(y) / y in y^2 by reweighted least squares); in fp32
//   3.6e-8.  (Degree 7: 1.3e-7, of which 2.3e-6 of a small score, which L shows; one
//   FMA less.)  It needs no special function, of which the other form takes 1 1/4.
// slope: with the polynomial's x (log2 units), a quarter of the derivative
// 1 - (x / log2c)^2 is 1/4 + slope x^2.
struct CapParams {
  float log2c, in, small2, a[5], slope;
};
inline CapParams cap_params(float softcap, float scale) {
  CapParams c = {};
  if (!(softcap > 0.f)) return c;
  const double b[5] = {0.9999999316224369, -0.3333277617751536, 0.13320570677476742, -0.05276213076364388,
                       0.016737567205032073};
  const double log2e = 1.4426950408889634, k = (double)scale / softcap;
  c.log2c = (float)(softcap * log2e);
  c.in = (float)(2.0 * scale * log2e / softcap);
  c.slope = (float)(-0.25 / ((double)softcap * log2e * softcap * log2e));
  // (past k = 1000, or with a scale past 2^20, the coefficients could leave fp32: the
  // first form then serves all)
  const bool fits = k < 1000.0 && scale < 0x1p20f;
  c.small2 = fits ? (float)(0.25 / (k * k)) : -1.f;
  double f = scale * log2e;
  for (int i = 0; i < 5; ++i, f *= k * k) c.a[i] = fits ? (float)(b[i] * f) : 0.f;
  return c;
}

// The cap's derivative is 4 r (1 - r); the kernels leave the 4 to this factor.
inline float scale_grad(const Problem& p, const ScoreMods& m) { return m.softcap > 0.f ? 4.f * p.scale : p.scale; }

// Few query rows over many keys (score-modified forward).
// Packing: the G query heads of a key/value head are G * Tq consecutive rows of Q, O
// and L, so a call of at most 64 query rows runs them as one head's rows: K and V
// are walked once for the group, in tiles that are at least as full.
// Splitting: where the work items fill at most half of the SMs, each item's key
// tiles are dealt to `split` CTAs.  Each leaves its unnormalised O, reference and
// sum (fp32) in the workspace, and a second kernel joins them.
constexpr int kPackRows = 64;
struct FwdShape {
  int heads, rows;  // per batch entry, rows per head
  int row_mod;      // packed: Tq, the period of the rows' positions; else 0
  int group;        // packed: G; else 1
  long long items;  // pairs of query tiles
  int split;        // CTAs per item
  bool few() const { return row_mod || split > 1; }
};
inline FwdShape fwd_shape(const Problem& p, const ScoreMods& m, int sms) {
  FwdShape s = {p.Hq, p.Tq, 0, 1, 0, 1};
  if (m.any() && p.G() > 1 && p.Tq <= kPackRows && (long long)p.G() * p.Tq <= (1 << 24)) {
    s.heads = p.Hkv;
    s.rows = p.G() * p.Tq;
    s.row_mod = p.Tq;
    s.group = p.G();
  }
  s.items = (long long)p.B * s.heads * ((s.rows + 2 * kTile - 1) / (2 * kTile));
  if (m.any() && s.items > 0 && 2 * s.items <= sms) {
    // Key tiles an item can see.  A tile takes ~1.5 us, the parts and their joining
    // 5 to 6: four tiles and more a part, of twelve at least.  (Tq 777, window 200,
    // at most 4 tiles: 15.8 us whole, 20.0 in three parts; Tq 32, Tk 8032: 124 us
    // whole, 23 in parts and packed.)
    const long long seen = p.window ? ((long long)p.window + 2 * kTile - 1) / kTile + 1 : p.kv_tiles();
    const long long tiles = seen < p.kv_tiles() ? seen : p.kv_tiles();
    const long long most = tiles >= 12 ? tiles / 4 : 1, want = sms / s.items;
    s.split = (int)(want < most ? want : most);
  }
  return s;
}
// fp32 workspace of a split forward: per item, part and row the O row, its reference
// m, its sum l (-1: no key tile, no O) and the sum that O is divided by.
inline size_t fwd_workspace_bytes(const Problem& p, const FwdShape& s) {
  return s.split > 1 ? (size_t)s.items * s.split * 2 * kTile * (p.dv + 4) * sizeof(float) : 0;
}

// Mask plan: what fa_mask_plan wrote for one set of dims, as int32 arrays.
// Rows and keys are padded to whole tiles per batch entry.
constexpr int kPlanCtas = 8;  // CTAs that plan one batch entry, each with a flag of its own
struct PlanView {
  // row i sees keys [row_lo, row_hi) (empty where row_hi <= row_lo); with the
  // flag by_key only those of its own document
  const int *row_lo, *row_hi, *q_doc, *k_doc;
  const int *kv_beg, *kv_end;          // key tiles a query tile visits
  const int *key_from, *key_to;        // key j is seen by rows [key_from, key_to), unless the flag by_row
  const int *m_beg, *m_end;            // query tiles a key tile visits
  const int *pair_order, *key_order;   // pairs of query tiles, and key tiles, of a batch entry: most work first
  const int *tile_doc_lo, *tile_doc_hi;  // least and greatest document of a key tile
  const int *by_key, *by_row;          // [B][kPlanCtas], any nonzero: set
};
struct PlanLayout {
  long long row_lo, row_hi, q_doc, k_doc, kv_beg, kv_end, key_from, key_to, m_beg, m_end, tile_doc_lo, tile_doc_hi,
      pair_order, key_order, by_key, by_row, total;  // offsets in ints
};
inline PlanLayout plan_layout(const Problem& p) {
  const long long qt = (long long)p.B * p.q_tiles(), kt = (long long)p.B * p.kv_tiles();
  long long at = 0;
  auto take = [&at](long long n) {
    const long long o = at;
    at += (n + 3) / 4 * 4;
    return o;
  };
  PlanLayout l;
  l.row_lo = take(qt * kTile);
  l.row_hi = take(qt * kTile);
  l.q_doc = take(qt * kTile);
  l.k_doc = take(kt * kTile);
  l.key_from = take(kt * kTile);
  l.key_to = take(kt * kTile);
  l.kv_beg = take(qt);
  l.kv_end = take(qt);
  l.m_beg = take(kt);
  l.m_end = take(kt);
  l.tile_doc_lo = take(kt);
  l.tile_doc_hi = take(kt);
  l.pair_order = take((long long)p.B * ((p.q_tiles() + 1) / 2));
  l.key_order = take(kt);
  l.by_key = take((long long)p.B * kPlanCtas);
  l.by_row = take((long long)p.B * kPlanCtas);
  l.total = at;
  return l;
}
inline PlanView plan_view(const Problem& p, const void* plan) {
  PlanView v = {};
  if (!plan) return v;
  const int* a = static_cast<const int*>(plan);
  const PlanLayout l = plan_layout(p);
  v.row_lo = a + l.row_lo;
  v.row_hi = a + l.row_hi;
  v.q_doc = a + l.q_doc;
  v.k_doc = a + l.k_doc;
  v.kv_beg = a + l.kv_beg;
  v.kv_end = a + l.kv_end;
  v.key_from = a + l.key_from;
  v.key_to = a + l.key_to;
  v.m_beg = a + l.m_beg;
  v.m_end = a + l.m_end;
  v.pair_order = a + l.pair_order;
  v.key_order = a + l.key_order;
  v.tile_doc_lo = a + l.tile_doc_lo;
  v.tile_doc_hi = a + l.tile_doc_hi;
  v.by_key = a + l.by_key;
  v.by_row = a + l.by_row;
  return v;
}
#ifdef __CUDACC__
__device__ __forceinline__ bool plan_flag(const int* flags, int batch) {
  const int4* f = reinterpret_cast<const int4*>(flags) + (size_t)batch * (kPlanCtas / 4);
  int any = 0;
#pragma unroll
  for (int c = 0; c < kPlanCtas / 4; ++c) {
    const int4 v = __ldg(f + c);
    any |= v.x | v.y | v.z | v.w;
  }
  return any != 0;
}
#endif

// Documents and prefixes of a mask plan (device arrays, any of them null).
struct MaskInputs {
  const int *doc_q, *doc_k;  // [B, Tq], [B, Tk]
  const int* prefix;         // [B], or [B, Tq] with prefix_per_row
  int prefix_per_row;
};
cudaError_t launch_mask_plan(const Problem& p, const MaskInputs& in, void* plan, cudaStream_t stream);

// Parameters of the backward main kernel.
struct BwdParams {
  const float* lse2;
  const float* delta;
  int* status;
  int Hq, Hkv, G, Tq, Tk, causal_off, q_tiles, kv_tiles;
  int sb_groups;  // (batch, kv head) groups per super-batch of the grid order; divides B * Hkv
  int window;     // causal sliding window in keys, 0 = none
  long long Tq_pad;
  float scale_log2, scale_grad;  // scale_grad: of dK (scale, times 4 with a cap)
  int test_withhold_do;  // test build only: never issue the dO loads (the CTA's waits then time out)
  // Split items.  Plain rule: the last n_split items of the grid order run as two
  // CTAs each (CTAs n_whole + 2 s and n_whole + 2 s + 1 for item n_whole + s), each
  // walking half of the item's query tiles.  Scored calls of few items
  // (ScoredBwdParams::split_first): the first n_split items run as `parts` CTAs each
  // (CTAs parts * s ... for item s), each walking its share; with a plan as many of
  // them as there is work for.  The CTAs' fp32 dK / dV meet in `part`, and whichever
  // finishes last adds them up (more than two: in their order) and stores the sum.
  // split_counters, zeroed by fa_bwd_pre, count those that have written theirs; in
  // scored calls the second of two that finds the first counted before it writes
  // neither writes nor counts.
  int n_whole, n_split;
  float* part;                    // [n_split][2, or parts][128 key rows][d + dv]
  unsigned int* split_counters;   // [n_split]
};
// What the score-modified instances need besides (see ScoreMods).
struct ScoredBwdParams : BwdParams {
  CapParams cap;
  const float* slopes;     // [Hq]
  int hi_off, lo_off;      // row i sees keys [i + lo_off, i + hi_off) (no plan)
  int two_sided;           // a row may see keys on both sides of its own position
  int parts, split_first;  // CTAs per split item (2 by the plain rule); whether those are the order's first (scored_split)
  PlanView plan;
};

// The score-modified instances, by head size of Q and K (one translation unit
// and direction each).
using FwdLauncher = cudaError_t (*)(const Problem& p, const ScoreMods& m, const FwdShape& s, const CUtensorMap& mq,
                                    const CUtensorMap& mk, const CUtensorMap& mv, void* O, float* L, float* part,
                                    cudaStream_t stream);
// For the problem's modifications and value head size; _few: with kFew.
FwdLauncher fwd_scored_64(const Problem& p, const ScoreMods& m);
FwdLauncher fwd_scored_128(const Problem& p, const ScoreMods& m);
FwdLauncher fwd_scored_few_64(const Problem& p, const ScoreMods& m);
FwdLauncher fwd_scored_few_128(const Problem& p, const ScoreMods& m);
cudaError_t launch_bwd_scored_64(const Problem& p, const ScoreMods& m, const CUtensorMap* maps, const ScoredBwdParams& bp,
                                 cudaStream_t stream);
cudaError_t launch_bwd_scored_128(const Problem& p, const ScoreMods& m, const CUtensorMap* maps, const ScoredBwdParams& bp,
                                  cudaStream_t stream);

// Launchers.  Each returns the first CUDA error it met and adds the number
// of kernels it enqueued to *launches.
cudaError_t launch_forward(const Problem& p, const ScoreMods& m, const void* Q, const void* K, const void* V, void* O,
                           float* L, void* workspace, size_t workspace_bytes, cudaStream_t stream, int* launches);
// `workspace_bytes` decides whether the split-item area fits (see BwdWorkspace).
cudaError_t launch_backward(const Problem& p, const ScoreMods& m, const void* Q, const void* K, const void* V, const void* O,
                            const void* dO, const float* L, void* dQ, void* dK, void* dV, void* workspace,
                            size_t workspace_bytes, int stages, cudaStream_t stream, int* launches);

// Groups per super-batch of the backward's grid order: the smallest divisor
// S of n_groups with S * kv_tiles >= 1.5 * sms, searched up to four times the
// least such S; n_groups (a single super-batch) when there is none.
inline int super_batch_groups(int n_groups, int kv_tiles, int sms) {
  if (n_groups < 1 || kv_tiles < 1) return n_groups;
  const long long want = (3LL * sms + 1) / 2;
  const long long s_min = want <= kv_tiles ? 1 : (want + kv_tiles - 1) / kv_tiles;
  for (long long s = s_min; s < n_groups && s <= 4 * s_min; ++s)
    if (n_groups % s == 0) return (int)s;
  return n_groups;
}

// The same with a mask plan, which knows each key tile's work.  Up to eight groups go as
// one super-batch, so that the heaviest tiles are the first of all; more groups' fp32 dQ
// and dO would no longer stay in L2, and within super-batches the tiles still go by work.
// Main kernel, one super-batch / the plain rule's, us, heads of 128 (query / kv heads),
// packed documents:
//   4 x T 8192, 8 / 2 of 64    238 / 270      B 1, T 8192, 40 / 10    393 / 371
//   B 1, T 16384, 32 / 4      1231 / 1286     B 1, T 8192, 48 / 12    465 / 471
//   B 1, T 8192, 32 / 8        303 / 330      B 2, T 4096, 32 / 8     211 / 195
//   B 1, T 32768, 32 / 8      4182 / 4196     B 4, T 8192, 32 / 8    1565 / 1243
//   B 1, T 8192, 64 / 8        715 / 678      B 8, T 8192, 32 / 8    3702 / 2438
// (one document: B 8 12082 / 8011, where the unmodified call takes 8100).
constexpr int kPlannedGroups = 8;
inline int planned_super_batch_groups(int n_groups, int kv_tiles, int sms) {
  return n_groups <= kPlannedGroups ? n_groups : super_batch_groups(n_groups, kv_tiles, sms);
}

// Work items of the backward main kernel that may be split (in two: see
// backward_split_items; in parts: scored_split); the workspace holds their fp32
// partial dK / dV.
constexpr int kMaxSplitItems = 128;

// Workspace carve-up of fa_backward (byte offsets, 256-aligned).  `part` and
// `counters` (the split items' partial dK / dV and their finish counters)
// are empty when no item can be split (a plain call with a causal mask, or a
// scored one of many items).  The backward needs `total_min` bytes (up to `part`); it splits items only when the
// workspace also holds the split area (`total`).
struct BwdWorkspace {
  size_t dq_acc, lse2, delta, part, counters, total_min, total;
  int split_cap;  // items the partial area has room for
};
// slots: rows of 128 keys in the partial area (items * parts); -1: the plain rule.
BwdWorkspace backward_workspace_layout(const Problem& p, long long slots = -1, int items = 0);

// Split items of the score-modified backward.  A key tile's work is the query tiles
// that see it, so where there are few items the heaviest alone can outlast the
// rest (a causal call with one item per SM runs twice its mean).  Then the items
// above the mean per SM, the first of the order, run in parts; four tiles are
// left to a part, whose set-up and fp32 partial sums cost about as much as two.
// (B 2, 16 / 4 heads of 128, T 2001, prefixes: 142 us whole, 114 with every item in
// four parts, 105 with the heavier half of the items in two; with all of them in two
// 97 out of L2, but the step's time on cold data rises by 7 for the partial sums.)
// With more than two items per SM the plain rule holds (equal work: a short last round
// in halves).
// What a plan hides is not known here; its items are split as they are without it, and
// in the kernel an item takes as many of its parts as have kPlannedPartTiles tiles: the
// mean is lower than was counted, so a part has to be worth more.  Backward, us, all
// parts / 4 tiles a part / 8 / 12 / 16 / nothing split; heads of 128:
//   4096 tokens in documents of 64, 8 / 2 heads        81   37   37   37   37   37
//   2048 in documents of 300, 16 / 4                   90   84   61   61   61   61
//   2 x 2001 in documents of 700, 16 / 4               92   92   91   84   86   87
//   2048 in documents of 1000, 8 / 1                  125  137  135  117  111  170
//   2048 in one document, 16 / 4                      109  119  115  109  109  158
constexpr int kPartTiles = 4, kPlannedPartTiles = 12;
struct ScoredSplit {
  int items, parts;  // 0: none
};
inline ScoredSplit scored_split(const Problem& p, int sms) {
  const long long groups = (long long)p.B * p.Hkv, n = groups * p.kv_tiles();
  if (n < 1 || sms < 1 || n > 2LL * sms || p.q_tiles() < 1) return {0, 1};
  const int hi = row_hi_off(p), lo = row_lo_off(p);
  auto work = [&](int k) {  // query tiles of key tile k, all heads of a group
    const int k0 = k * kTile, last_key = (k0 + kTile < p.Tk ? k0 + kTile : p.Tk) - 1;
    const int first = k0 - hi + 1 > 0 ? (k0 - hi + 1) / kTile : 0, last_row = last_key - lo;
    const int end = last_row < 0 ? 0 : last_row / kTile + 1 < p.q_tiles() ? last_row / kTile + 1 : p.q_tiles();
    return end > first ? (long long)p.G() * (end - first) : 0LL;
  };
  long long total = 0, most = 0;
  for (int k = 0; k < p.kv_tiles(); ++k) {
    const long long w = work(k);
    total += w * groups;
    if (w > most) most = w;
  }
  const double mean = (double)total / sms, target = mean > kPartTiles ? mean : kPartTiles;
  int parts = (int)(most / (1.2 * target)) + (most > 1.2 * target);
  if (parts > 8) parts = 8;
  long long items = 0;
  for (int k = 0; k < p.kv_tiles() && (double)work(k) > target; ++k) items += groups;
  if (items > kMaxSplitItems) items = kMaxSplitItems;
  return parts < 2 || items < 1 ? ScoredSplit{0, 1} : ScoredSplit{(int)items, parts};
}

}  // namespace fa
