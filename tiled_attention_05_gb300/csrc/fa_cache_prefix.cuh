// Attention of many rows over one shared prefix (fa_cache_attention): the rows of all
// sequences of a group meet the prefix's keys at once, on the tcgen05 tensor cores.
// What comes out are parts (unnormalised O, reference, sum) that the join adds to those
// of the sequences' own keys.
//
// An item is (group, kv head, up to 256 rows), two tiles of 128; the list of items times
// key tiles of 128 is cut into equal shares, one CTA an SM each.  Two tiles of rows and 128
// keys take ~3300 cycles, where the MMAs alone take ~2200 (some 64 each, the tensor pipe's own
// time): the MMA thread bounds it, by its commits (some 150 each) and waits.  In e4m3 they take
// ~5400: the chain of a tile's softmax (2400) and of its turn on the MMA thread.  Measured (32 / 8
// heads of 128): 1024 rows over 32768 keys of bf16, on the ~105 SMs that the own keys leave, 151 us;
// 256 over 8192 in e4m3, 34 us, some 10 of them until the first scores.  Roles:
//   warp 0       issues the MMAs of both tiles in turn, S_X(j) = Q_X K_j^T and
//                O_X += P_X(j) V_j, so that the tensor pipe runs one tile's while the
//                softmax works on the other's (the forward's order: those of one
//                thread execute in issue order, so S_X(j + 1) may overwrite P_X(j))
//   warps 1..3   bring K_j and V_j from their pages into the ring's slots: bf16 by TMA, a
//                box a page (by cp.async of these warps, 16 bytes a lane, a tile took them
//                4 us); e4m3 by bulk copies into raw buffers, which the three warps
//                turn into fp16 in the swizzle that TMA writes
//   warps 4..11  softmax of tile A and of tile B, a thread a row: scores from TMEM, exp2, P
//                as 16-bit pairs over the scores, O rescaled in TMEM when the maximum grows
//                by more than 2^8; before that the row of Q into shared memory, after
//                it the part to the workspace.  bf16: the row's scores in registers.
//                e4m3 and capped: two passes of 32 columns over TMEM, whose code is a
//                quarter as long (short calls run it cold)
//   dual         an item of at most 128 rows: both tiles are its rows, A over the even key tiles
//                and B over the odd ones, with a part each
// bf16: a weight is one bf16, as in the forward: O is 2.3e-3 from 64 bits over 32768 keys, where the
// result's own rounding is 1.7e-3.  (Two of them, as in fa_cache_attn.cuh, where HBM leaves the
// time, would be half as many MMAs again for the thread that bounds this kernel.)
// e4m3: as in fa_cache_attn.cuh, codes and weights meet in fp16, the key's scale
// multiplies the score, the value's goes into the exponent.  (Codes could feed the fp8
// pipe as they are, but then the weights would be e4m3 too: a sum of two has a weight's
// 8 bits, and ends at 2^-18 of the largest, which a long flat tail falls below.)
// MODS: kLines, slopes or a window (bf16), or kCapped, a cap, with or without these.  (With the cap
// in the registers' form too, its code for each four columns made a prefix with slopes alone
// take 70 us for 39.)
// WINDOW: the call has one.  (Its code in all of them, though jumped over, made a prefix with slopes
// alone take 48.5 us for 47.2: 16 answers to each of 8 prompts.)
#pragma once
#include <climits>
#include <cstdint>
#include <type_traits>

#include "fa_cache_internal.h"
#include "sm103_ptx.cuh"

namespace {

using namespace fa_ptx;
using fa::CacheEntry;
using fa::CacheParams;

constexpr int kThreads = 384, kLoaders = 96;  // (three warps of them load)
constexpr int BM = 128, BN = fa::kPrefixKeys;
enum : int { kUnmodified = 0, kLines = 1, kCapped = 2 };
// Register split, as in the forward: 88 + 2 * 208 = 3 * 168.
constexpr int kRegsLaunch = 168, kRegsLow = 88, kRegsHigh = 208;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: weights stay <= 256

template <int D, int DV, bool Q8>
struct PrefixCfg {
  static constexpr int W = D > DV ? D : DV;
  static constexpr int Q_BYTES = BM * D * 2, SLOT = BN * W * 2;
  static constexpr int RAW = Q8 ? BN * W : 0;  // a slot's codes
  static constexpr int NRAW = Q8 ? 3 : 0;
  static constexpr int SCALES = Q8 ? 2 * 2 * 3 * BN * 4 : 0;  // [tile][buffer][k_scale, log2 v_scale, 1 / v_scale][key]
  static constexpr int OFF_SLOT = 2 * Q_BYTES;
  static constexpr int ROOM = (226 << 10) - 1024 - OFF_SLOT - NRAW * RAW - SCALES;
  static constexpr int NS = ROOM / SLOT > 6 ? 6 : ROOM / SLOT;
  static constexpr int OFF_RAW = OFF_SLOT + NS * SLOT;
  static constexpr int OFF_SCALES = OFF_RAW + NRAW * RAW;
  static constexpr int OFF_BAR = OFF_SCALES + SCALES;
  static constexpr int OFF_ROW = OFF_BAR + 256;  // (the barriers take 8 (2 NS + 19) + 8 bytes)
  static constexpr int OFF_SEEN = OFF_ROW + 256;
  static constexpr int SMEM = OFF_SEEN + (Q8 ? 0 : 2 * (DV + 1) * 4);
  // The softmax looks for V_j and K_{j+1} on the MMA thread's behalf (256 answers to 32768 tokens
  // 165 us, 168 without), unless slots are few: then it would wait for a K that is late.
  static constexpr bool VOUCHED = NS > 4;
  // (V_j leaves its slot after S_A(j + 1): K_{j+1} needs another one)
  static_assert(NS >= 3 && NS <= 6 && SMEM <= (226 << 10), "shared memory");
};

// Instruction descriptor, kind::f16 with fp32 D; A and B fp16 or bf16.
__host__ __device__ constexpr uint32_t idesc(bool f16, int M, int N, int b_mn) {
  return f16 ? idesc_bf16(M, N, 0, b_mn) & ~((1u << 7) | (1u << 10)) : idesc_bf16(M, N, 0, b_mn);
}
__device__ __forceinline__ uint32_t half2_of(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 c, u;\n\tmov.b32 {c, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}
// Four capped scores in log2 units (see CapParams): by the polynomial where that serves all
// of the warp's, else by the form for any.
__device__ __forceinline__ void cap_quad_of(const fa::CapParams& c, uint64_t& a, uint64_t& b) {
  const uint64_t ua = f2_mul(a, a), ub = f2_mul(b, b);
  const float top = fmax3(fmaxf(f2_lo(ua), f2_hi(ua)), f2_lo(ub), f2_hi(ub));
  if (__any_sync(~0u, !(top <= c.small2))) {
    uint64_t r0, r1, e0, e1;
    const uint64_t in = f2_pack(c.in, c.in), scale = f2_pack(-2.f * c.log2c, -2.f * c.log2c), top2 = f2_pack(c.log2c, c.log2c);
    cap_quad<true>(f2_mul(a, in), f2_mul(b, in), r0, r1, e0, e1);
    a = f2_fma(r0, scale, top2);
    b = f2_fma(r1, scale, top2);
    return;
  }
  uint64_t ta = f2_pack(c.a[4], c.a[4]), tb = ta;
#pragma unroll
  for (int k = 3; k >= 0; --k) ta = f2_fma(ta, ua, f2_pack(c.a[k], c.a[k])), tb = f2_fma(tb, ub, f2_pack(c.a[k], c.a[k]));
  a = f2_mul(a, ta);
  b = f2_mul(b, tb);
}

// bf16 with a window: a NaN or an infinity among the values of a tile reaches rows that do not see it,
// through their weights of 0.  A CTA in whose results is one says so in the workspace, and the kernel
// after it (CAREFUL), whose other CTAs end at once, goes through that share again: in
// tiles that not all rows see whole it replaces such values by 0, and notes the last key with one
// in each channel.  A row sees a prefix from some key on to its end, so that this key says
// whether it saw any: then its result there is NaN.  (64 answers of 16 to 1000 to 8192 tokens,
// window 4096: 66 us, 101 with the loader looking for them at once, 68 without any of this; 16 to each of
// 8 prompts of 2001, heads of 64, window 1000: 59, 94 and 56.)
template <int D, int DV, bool Q8, int MODS, bool WINDOW, bool CAREFUL>
__global__ void __launch_bounds__(kThreads, 1)
    fa_cache_prefix_kernel(const CacheParams p, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using C = PrefixCfg<D, DV, Q8>;
  using Cursor = fa::CacheCursor<BN, fa::kPrefixRows, fa::kPrefixItem, WINDOW>;
  constexpr int NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Cursor s_walk[9];
  constexpr bool kLooks = !Q8 && WINDOW && !CAREFUL;
  grid_next();  // the own keys' kernel, on the SMs that this one leaves
  if constexpr (CAREFUL) {
    grid_previous();
    if (p.look[blockIdx.x] == 0) return;
  }
  const auto share = fa::cache_share<BN, fa::kPrefixRows, fa::kPrefixItem, kThreads, WINDOW>(p);
  if (share.begin >= share.end || share.start.at >= share.end) {
    if (kLooks && threadIdx.x == 0) p.look[blockIdx.x] = 0;
    return;
  }

  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [NS] a slot holds its tile
  uint64_t* empty = full + NS;     // [NS]
  uint64_t* q_full = empty + NS;   // [2]
  uint64_t* s_full = q_full + 2;   // [2]
  uint64_t* p_full = s_full + 2;   // [2]
  uint64_t* o_done = p_full + 2;   // [2]
  uint64_t* raw_full = o_done + 2;    // [3] a raw buffer holds its codes (bf16: [0], a tile's rows have come, before zeros go to some)
  uint64_t* raw_empty = raw_full + 3;  // [3]
  uint64_t* found_full = raw_empty + 3;    // [2] see found_of
  uint64_t* found_free = found_full + 2;   // [2]
  uint64_t* drain = found_free + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* s_row = smem + C::OFF_ROW;
  // CAREFUL: two buffers, for items in turn, of the last key with a NaN or an infinity in each channel,
  // and behind the channels the number of them.
  auto found_of = [&](int item) { return reinterpret_cast<int*>(smem + C::OFF_SEEN) + (item & 1) * (DV + 1); };
  volatile int* not_finite = found_of(0);  // (not CAREFUL) a row's result has a NaN or an infinity
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    *abort_flag = (smem_u32(smem) & 1023u) ? 1 : 0;  // swizzled tiles need 1024 B alignment
    if (kLooks) *not_finite = 0;
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], Q8 ? kLoaders / 32 : 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 3; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], kLoaders / 32);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 128);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 128);
      mbar_init(&o_done[x], 1);
      mbar_init(&found_full[x], 1);
      mbar_init(&found_free[x], 256);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool run = *abort_flag == 0;
  const int page_mask = (1 << p.page_log2) - 1;

  // The items of the share: [c0, c1) are the key tiles of one.
  struct Item {
    int c0, c1;
  };
  auto item_of = [&](const Cursor& it) {
    return Item{it.c, it.end(p, share.end)};
  };
  // Whether tile B has rows of its own.  Where it has none, it takes the same rows as tile A, A
  // the item's even key tiles and B its odd ones; both leave a part.
  auto first_row = [&](const Cursor& it) { return (it.r * it.bundle + share.tile) * fa::kPrefixRows; };
  auto two_tiles = [&](const Cursor& it) { return it.n.rows > first_row(it) + BM; };

  if (warp < 4) {
    setmaxnreg_dec<kRegsLow>();
    if (warp == 0) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0 && run) {
        constexpr uint32_t idS = idesc(Q8, BM, BN, 0), idPV = idesc(Q8, BM, DV, 1);
        const uint32_t q_buf = smem_u32(smem), slots = smem_u32(smem + C::OFF_SLOT);
        // Slots and phases of the next K and the next V to read: every other unit of the ring.
        int sk = 0, sv = 1;
        uint32_t pk = 0, pv = 0, nq[2] = {0, 0}, np[2] = {0, 0};
        auto pass = [](int& s, uint32_t& phase) {
          s += 2;
          if (s >= NS) s -= NS, phase ^= 1;
        };
        const uint64_t q_desc = desc_kmajor(q_buf), k_desc = desc_kmajor(slots), v_desc = desc_mnmajor(slots, BN * 128);
        bool ok = true;
        // S_X of the next K; `first`: of the item, whose Q has to be there; `wait`: nobody has
        // looked for the K (or V); `last`: this tile is the last to read it.  Every check of a
        // barrier costs the tensor pipe a round trip (see VOUCHED).
        auto issue_s = [&](int x, bool first, bool wait, bool last) -> bool {
          if (first) {
            if (!mbar_wait_for(&q_full[x], nq[x], abort_flag)) return false;
            nq[x] ^= 1;
          }
          if (wait && !mbar_wait_for(&full[sk], pk, abort_flag)) return false;
          tc_fence_after();
          const uint64_t a0 = desc_at(q_desc, x * C::Q_BYTES), b0 = desc_at(k_desc, sk * C::SLOT);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k >> 2) * (BM * 128) + (k & 3) * 32;
            mma_ss(tmem + x * 128, desc_at(a0, off), desc_at(b0, off), idS, k > 0 ? 1u : 0u);
          }
          mma_commit(&s_full[x]);
          if (last) {
            mma_commit(&empty[sk]);
            pass(sk, pk);
          }
          return true;
        };
        auto issue_pv = [&](int x, bool first, bool wait, bool last) -> bool {
          if (!mbar_wait_for(&p_full[x], np[x], abort_flag)) return false;
          np[x] ^= 1;
          if (wait && !mbar_wait_for(&full[sv], pv, abort_flag)) return false;
          tc_fence_after();
          const uint64_t v0 = desc_at(v_desc, sv * C::SLOT);
#pragma unroll
          for (int k = 0; k < BN / 16; ++k)
            mma_ts(tmem + 256 + x * 128, tmem + x * 128 + k * 8, desc_at(v0, k * 2048), idPV, !first || k > 0 ? 1u : 0u);
          if (last) {
            mma_commit(&empty[sv]);
            pass(sv, pv);
          }
          return true;
        };
        Cursor* const walk = &s_walk[8];
        *walk = share.start;
        while (ok && walk->at < share.end) {
          const int tiles = walk->end(p, share.end) - walk->c;
          const bool two = two_tiles(*walk);
          // tile B's first key tile, and the distance of a tile's next one
          const int step = two ? 1 : 2, first_b = two ? 0 : 1;
          ok = issue_s(0, true, true, !two) && (first_b >= tiles || issue_s(1, true, !two, true));
          for (int j0 = 0; ok && j0 < tiles; j0 += step) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int j = x ? j0 + first_b : j0;
              if (j >= tiles || !ok) break;
              const bool mine = x == 0 || !two, last = x == 1 || !two;
              ok = issue_pv(x, j0 == 0, !C::VOUCHED && mine, last);
              if (!ok) break;
              if (j + step < tiles)
                ok = issue_s(x, false, C::VOUCHED ? !two : mine, last);
              else
                mma_commit(&o_done[x]);
            }
          }
          walk->next(p);
        }
        // Let every MMA issued above finish before TMEM is released.
        mma_commit(drain);
        mbar_wait_bounded(drain, 0);
      }
    } else {
      // ------------------------------------------------------------ loaders
      // Units K_0, V_0, K_1, ... of all items; unit u goes to slot u % NS (e4m3: by way of the
      // raw buffer u % NRAW).  Warp 1 issues the copies, a page (or 128 rows of it) a lane.
      const int tid = threadIdx.x - 32;
      uint8_t* slots = smem + C::OFF_SLOT;
      const int box = p.page_log2 < 7 ? 1 << p.page_log2 : BN;  // rows of a copy
      struct Units {
        Cursor it;
        Item m;
        int c, u;
        bool v;
      };
      auto step = [&](Units& n) {  // to the next unit; false at the share's end
        ++n.u;
        n.v = !n.v;
        if (n.v || ++n.c < n.m.c1) return true;
        n.it.next(p);
        if (n.it.at >= share.end) return false;
        n.m = item_of(n.it);
        n.c = n.m.c0;
        return true;
      };
      Units ld = {share.start, item_of(share.start), 0, 0, false};
      ld.c = ld.m.c0;
      bool ok = run;
      // The page of this lane's 16 rows of a tile: -1 if no row of it is needed (it ends before the
      // first key that is seen, or begins behind the last), -2 if it does not fit.
      int id = 0;
      auto fetch_id = [&]() {
        const int key = (ld.it.n.chunk0 + ld.c) * BN + (lane & 7) * 16;
        id = -1;
        if (key >= ld.it.n.keys || (WINDOW && (key | page_mask) < ld.it.n.from)) return;
        id = __ldg(p.p_tables + (long long)ld.it.e * p.p_cols + (key >> p.page_log2));
        if ((unsigned)id >= (unsigned)p.pages) fa::cache_bad(p.status), id = -2;
      };
      // Copies of unit ld; `bar` gets their bytes.
      auto copy = [&](uint64_t* bar, uint8_t* dst) {
        const int row = (lane & 7) * 16, width = ld.v ? DV : D;
        const bool mine = lane < 8 && row % box == 0 && id >= 0;
        const unsigned all = __ballot_sync(~0u, mine);
        if constexpr (Q8) {  // codes that a bad page leaves out are 0
          if (lane < 8 && id == -2) {
#pragma unroll 1
            for (int k = 0; k < width; ++k) st_shared_v4(smem_u32(dst + row * width) + k * 16, 0, 0, 0, 0);
            fence_async_smem();
          }
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(all) * box * width * (Q8 ? 1 : 2));
        __syncwarp();
        if (!mine) return;
        const int at = ((ld.it.n.chunk0 + ld.c) * BN + row) & page_mask;
        const int head = id * p.Hkv + ld.it.h;
        if constexpr (Q8) {
          bulk_load(dst + row * width, (ld.v ? p.V : p.K) + (((long long)head << p.page_log2) | at) * width, box * width, bar);
        } else {
          for (int cb = 0; cb < width / 64; ++cb)
            tma_load_3d(dst + cb * (BN * 128) + row * 128, ld.v ? &tmV : &tmK, bar, cb * 64, at, head);
        }
      };
      if constexpr (!Q8) {
        if (warp == 1) {
          int zeroed = 0;  // tiles of values, in whose rows zeros are written
          int items = 0, all_from = 0;  // of the share so far; first key that all rows of the item's group see
          bool more = true;
          auto begin_item = [&]() {
            if (!__all_sync(~0u, mbar_wait_for(&found_free[items & 1], ((items >> 1) & 1) ^ 1, abort_flag))) return false;
            int* found = found_of(items);
            for (int k = lane; k <= DV; k += 32) found[k] = k < DV ? -1 : 0;
            int first, end, most = 0;
            fa::cache_group(p, ld.it.e, &first, &end);
            for (int b = first + lane; b < end; b += 32) most = max(most, fa::cache_length(p, b));
            all_from = ld.it.n.keys + __reduce_max_sync(~0u, most) - p.window;  // (the furthest row is the last of the longest)
            __syncwarp();
            return true;
          };
          fetch_id();
          while (ok && more) {
            if (CAREFUL && !ld.v && ld.c == ld.m.c0 && !begin_item()) break;
            const int s = ld.u % NS, valid = ld.it.n.keys - (ld.it.n.chunk0 + ld.c) * BN;
            if (!__all_sync(~0u, mbar_wait_for(&empty[s], ((ld.u / NS) & 1) ^ 1, abort_flag))) break;
            // Rows past the prefix's end or before the first key that is seen, whatever the pages hold
            // there, and what a page that was not copied leaves from an earlier tile: as keys they
            // meet a score that is masked, as values a weight of 0, for which they have to be finite.
            const int first = WINDOW ? ld.it.n.from - (ld.it.n.chunk0 + ld.c) * BN : 0;
            const unsigned bad = __ballot_sync(~0u, lane < 8 && id == -2);  // blocks of 16 rows
            const int all = CAREFUL ? min(all_from - (ld.it.n.chunk0 + ld.c) * BN, min(valid, BN)) : 0;
            const bool look = ld.v && (valid < BN || first > 0 || bad || all > 0);
            copy(look ? raw_full : &full[s], slots + s * C::SLOT);
            if (look) {
              ok = __all_sync(~0u, mbar_wait_for(raw_full, zeroed++ & 1, abort_flag));
              auto zero = [&](int row0, int row1) {
                for (int k = lane; k < (row1 - row0) * (DV / 8); k += 32) {
                  const int row = row0 + k / (DV / 8), chunk = k % (DV / 8);
                  st_shared_v4(smem_u32(slots + s * C::SLOT) + (chunk >> 3) * (BN * 128) + sw128_offset(row, chunk & 7), 0, 0, 0, 0);
                }
              };
              zero(0, first);
              zero(valid, BN);
#pragma unroll 1
              for (unsigned b = bad; b; b &= b - 1) zero((__ffs(b) - 1) * 16, __ffs(b) * 16);
              if constexpr (CAREFUL) {  // rows that some of the item's do not see
                __syncwarp();
                int* found = found_of(items);
#pragma unroll 4
                for (int k = max(first, 0) * (DV / 8) + lane; k < all * (DV / 8); k += 32) {
                  const int row = k / (DV / 8), chunk = k % (DV / 8);
                  const uint32_t at = (chunk >> 3) * (BN * 128) + sw128_offset(row, chunk & 7);
                  const float4 v = ld_shared_f4(slots + s * C::SLOT + at);
                  const uint32_t w[4] = {__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w)};
                  uint32_t b[4];
#pragma unroll
                  for (int y = 0; y < 4; ++y) b[y] = not_finite2(w[y]);
                  if (!(b[0] | b[1] | b[2] | b[3])) continue;
                  st_shared_v4(smem_u32(slots + s * C::SLOT) + at, w[0] & ~b[0], w[1] & ~b[1], w[2] & ~b[2], w[3] & ~b[3]);
                  atomicAdd(&found[DV], 1);
#pragma unroll 1
                  for (int y = 0; y < 8; ++y)
                    if ((b[y >> 1] >> (16 * (y & 1))) & 1u) atomicMax(&found[chunk * 8 + y], (ld.it.n.chunk0 + ld.c) * BN + row);
                }
              }
              fence_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&full[s]);
            }
            if (CAREFUL && ld.v && ld.c + 1 == ld.m.c1) {  // all of the item's values have been looked at
              __syncwarp();
              if (lane == 0) mbar_arrive(&found_full[items & 1]);
              ++items;
            }
            more = step(ld);
            if (more && !ld.v) fetch_id();
          }
          // Copies in flight have to land before the CTA leaves its shared memory.
          if (zeroed) mbar_wait_bounded(raw_full, (zeroed - 1) & 1);  // (its slot's barrier was passed on by hand)
          for (int u = ld.u > NS ? ld.u - NS : 0; u < ld.u; ++u) mbar_wait_bounded(&full[u % NS], (u / NS) & 1);
        }
      } else {
        // e4m3: all three warps turn the codes of a raw buffer into fp16, pieces of 16 codes, four at
        // a time (a row has 1 << shift pieces).
        auto convert = [&](int shift, int first, int valid, const uint8_t* src, uint32_t dst) {
#pragma unroll 1
          for (int i0 = tid; i0 < BN << shift; i0 += 4 * kLoaders) {
            uint4 c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int i = i0 + k * kLoaders;
              c[k] = make_uint4(0, 0, 0, 0);
              if (i >= first << shift && i < valid << shift) c[k] = reinterpret_cast<const uint4*>(src)[i];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int i = i0 + k * kLoaders, row = i >> shift, piece = i - (row << shift);
              if (row >= BN) break;
              const uint32_t to = dst + (piece >> 2) * (BN * 128) + sw128_offset(row, (piece & 3) * 2);
              st_shared_v4(to, half2_of(c[k].x), half2_of(c[k].x >> 16), half2_of(c[k].y), half2_of(c[k].y >> 16));
              st_shared_v4(to ^ 16, half2_of(c[k].z), half2_of(c[k].z >> 16), half2_of(c[k].w), half2_of(c[k].w >> 16));
            }
          }
        };
        constexpr int NR = C::NRAW + !Q8;
        bool more_ld = true, more = true;
        auto issue = [&]() {  // (warp 1) the next unit's codes into their raw buffer
          if (warp != 1 || !more_ld || !ok) return;
          const int s = ld.u % NR;
          if (!__all_sync(~0u, mbar_wait_for(&raw_empty[s], ((ld.u / NR) & 1) ^ 1, abort_flag))) {
            ok = false;
            return;
          }
          copy(&raw_full[s], smem + C::OFF_RAW + s * C::RAW);
          more_ld = step(ld);
          if (more_ld && !ld.v) fetch_id();
        };
        fetch_id();
        Units now = ld;
#pragma unroll 1
        for (int k = 0; k < NR - 1; ++k) issue();
        while (ok && more) {
          issue();
          const int s = now.u % NS, rs = now.u % NR, valid = min(now.it.n.keys - (now.it.n.chunk0 + now.c) * BN, BN);
          const bool both = mbar_wait_for(&raw_full[rs], (now.u / NR) & 1, abort_flag) &&
                            mbar_wait_for(&empty[s], ((now.u / NS) & 1) ^ 1, abort_flag);
          if (!__all_sync(~0u, both)) break;
          const uint8_t* src = smem + C::OFF_RAW + rs * C::RAW;
          const uint32_t dst = smem_u32(slots + s * C::SLOT);
          const int first = WINDOW ? max(now.it.n.from - (now.it.n.chunk0 + now.c) * BN, 0) : 0;
          convert((now.v ? DV : D) == 128 ? 3 : 2, first, valid, src, dst);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full[s]);
            mbar_arrive(&raw_empty[rs]);
          }
          more = step(now);
        }
        if (warp == 1)
          for (int u = ld.u > NR ? ld.u - NR : 0; u < ld.u; ++u) mbar_wait_bounded(&raw_full[u % NR], (u / NR) & 1);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax of tile x
    setmaxnreg_inc<kRegsHigh>();
    const int x = (warp - 4) >> 2, quad = warp & 3, r = quad * 32 + lane;  // r: row inside the tile == TMEM lane
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_base, tO = tmem + 256 + x * 128 + lane_base;
    const float NEG_INF = -__int_as_float(0x7f800000);
    int ns = 0, no = 0, nb = 0;  // phases waited for; scale buffers written
    int units = 0;               // ring position of the item's first K
    [[maybe_unused]] int items = 0;  // of the share so far
    bool ok = run;
    // Loads from TMEM are a warp's, and the barrier that hands the scales round is the
    // tile's: those who meet there leave together when one of them gave up.
    auto agree = [&](bool fine) { return Q8 ? named_bar_and(1 + x, 128, fine) : (bool)__all_sync(~0u, fine); };
    // Where the walk stands, and what is left to say of this thread's row at an item's end, lie
    // in shared memory: the loop over an item's tiles needs the registers.
    Cursor* const walk = &s_walk[warp - 4];
    if (lane == 0) *walk = share.start;
    __syncwarp();
    while (ok && walk->at < share.end) {
      {
        const Cursor it = *walk;
        const bool two = two_tiles(it);
        const Item m = item_of(it);
        const int step = two ? 1 : 2, c0 = two ? m.c0 : m.c0 + x;  // this tile's key tiles: every step-th from c0 on
        const int tiles = (m.c1 - c0 + step - 1) / step;
        const int row = first_row(it) + (two ? x * BM : 0) + r;
        const fa::CacheRow w = fa::cache_row(p, it.n, row);
        const int head = it.h * p.G + w.g;
        float unit = MODS && p.capped ? 1.f : p.scale_log2;
        int lim = it.n.keys - (it.n.chunk0 + c0) * BN;  // columns of the next tile that are keys
        int pos = 0;  // of this row among the own keys; negative: padding
        float slope = 0.f;
        if (tiles > 0) {  // the warp's 32 rows of Q into shared memory
          constexpr int P = D / 8, STEP = 32 / P;  // lanes a row, rows at a time
          const int mine = w.valid ? (w.b * p.Hq + head) * p.T + w.t : -1, piece = lane % P;
          const uint32_t dst = smem_u32(smem) + x * C::Q_BYTES;
#pragma unroll 2
          for (int k = 0; k < 32; k += STEP) {
            const int from = __shfl_sync(~0u, mine, k + lane / P), row = quad * 32 + k + lane / P;
            cp16(dst + (piece >> 3) * (BM * 128) + sw128_offset(row, piece & 7), p.Q + (from < 0 ? 0ll : (long long)from * D + piece * 8),
                 from >= 0);
          }
          cp_commit();
          pos = fa::cache_length(p, w.b) - p.T + w.t;
          if (MODS && p.slopes) slope = __ldg(p.slopes + head) * 1.4426950408889634f;
          cp_wait<0>();
          if constexpr (Q8) {  // as fp16, a row's largest value brought to [1, 2); a row a thread
            __syncwarp();
            uint32_t top = 0;
#pragma unroll 2
            for (int k = 0; k < P; ++k) {
              const float4 v = ld_shared_f4(smem + x * C::Q_BYTES + (k >> 3) * (BM * 128) + sw128_offset(r, k & 7));
              const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int y = 0; y < 4; ++y)
                top = max(top, max(__float_as_uint(a[y]) & 0x7fffu, (__float_as_uint(a[y]) >> 16) & 0x7fffu));
            }
            const int ex = min(max((int)(top >> 7), 1), 253);
            const float down = __uint_as_float((uint32_t)(254 - ex) << 23);
            unit *= __uint_as_float((uint32_t)ex << 23);
#pragma unroll 2
            for (int k = 0; k < P; ++k) {
              const uint32_t at = (k >> 3) * (BM * 128) + sw128_offset(r, k & 7);
              const float4 v = ld_shared_f4(smem + x * C::Q_BYTES + at);
              uint32_t a[4] = {__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w)};
#pragma unroll
              for (int y = 0; y < 4; ++y)
                a[y] = pack_f16x2(__uint_as_float(a[y] << 16) * down, __uint_as_float(a[y] & 0xffff0000u) * down);
              st_shared_v4(dst + at, a[0], a[1], a[2], a[3]);
            }
          }
          fence_async_smem();
          mbar_arrive(&q_full[x]);
        }
        {
          s_row[threadIdx.x - 128] = !w.valid ? 0 : pos < 0 ? 2 : 1;  // 2: a padding row, whose part is none
        }
        // The scales of a tile's keys, one key a thread, a tile ahead.
        float ks = 0.f, vs = 0.f;
        auto fetch_scales = [&](int c) {
          const Cursor& it = *walk;
          const int key = (it.n.chunk0 + c) * BN + r;
          ks = 0.f, vs = 1.f;
          if (key >= it.n.keys || (WINDOW && key < it.n.from)) return;
          const int id = __ldg(p.p_tables + (long long)it.e * p.p_cols + (key >> p.page_log2));
          if ((unsigned)id >= (unsigned)p.pages) return;
          const long long at = (((long long)id * p.Hkv + it.h) << p.page_log2) | (key & page_mask);
          ks = __ldg(p.k_scale + at);
          vs = __ldg(p.v_scale + at);
        };
        if (Q8 && tiles > 0) fetch_scales(c0);
        float m_ref = NEG_INF, l = 0.f;
        for (int j = 0; ok && j < tiles; ++j) {
          const float* sc = nullptr;
          if constexpr (Q8) {
            float* to = reinterpret_cast<float*>(smem + C::OFF_SCALES) + (x * 2 + (nb & 1)) * 3 * BN;
            ++nb;
            const float a = lg2(fmaxf(vs, 0x1p-69f));  // (see fa_cache_attn.cuh)
            // A key's scale of NaN comes in with the value's, behind the cap and before the mask: the
            // cap would give it to the other keys of its four, hidden or not.
            const bool finite = fabsf(ks) < INFINITY;
            to[r] = finite ? ks : 0.f;
            to[BN + r] = finite && vs == vs ? a : __int_as_float(0x7fffffff);
            to[2 * BN + r] = ex2(-a);
            sc = to;
            if (j + 1 < tiles) fetch_scales(c0 + (j + 1) * step);
          }
          ok = mbar_wait_for(&s_full[x], ns & 1, abort_flag);
          ok = agree(ok);
          if (!ok) break;
          ++ns;
          tc_fence_after();
          // V_j and K_{j+1}, on behalf of the MMA thread: tile A looks for both.  (Not for a K where
          // the tiles have key tiles of their own: the next one may need the slot of V_j, which
          // this tile's P has to free first.)
          bool there = true;
          if (C::VOUCHED && r == 0 && (x == 0 || step == 2)) {
            const int at = units + 2 * ((step == 2 ? x : 0) + j * step);
            there = mbar_wait_for(&full[(at + 1) % NS], ((at + 1) / NS) & 1, abort_flag) &&
                    (step == 2 || j + 1 >= tiles || mbar_wait_for(&full[(at + 2) % NS], ((at + 2) / NS) & 1, abort_flag));
          }
          __syncwarp();
          float mt = NEG_INF, m_new, base, sum;
          bool rescale, warp_rescale;
          auto refer = [&]() {  // the reference of this tile's weights, from its maximum
            m_new = mt > m_ref + kRescaleThreshold ? mt : m_ref;  // also taken when m_ref == -inf
            rescale = j > 0 && m_new != m_ref && m_ref != NEG_INF;
            warp_rescale = __any_sync(~0u, rescale);
            base = m_new == NEG_INF ? 0.f : m_new;
          };
          if constexpr (Q8 || MODS == kCapped) {
            // Two passes of 32 columns at a time: the scores in log2 units, back into TMEM, and
            // their maximum; then the weights.  (With the row in registers the code is four
            // times as long, and short calls run it cold.)
            float top[2] = {NEG_INF, NEG_INF};
#pragma unroll 1
            for (int c = 0; c < BN; c += 32) {
              uint32_t s[32];
              tmem_ld32(tS + c, s);
              tmem_wait_ld();
              const uint64_t unit2 = f2_pack(unit, unit);
              const float far0 = (float)(pos + lim - c);  // of column c
              // Of the columns only those from `from` on and before `to` count.
              const int from = WINDOW ? pos + lim - c - p.window + 1 : 0, to = lim - c;
              const bool some_hidden = from > 0 || to < 32;
              if (MODS && some_hidden) {  // (a NaN there would reach the others of its four through the cap)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (e < from || e >= to) s[e] = 0u;
              }
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                uint64_t t[2] = {f2_mul(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), unit2),
                                 f2_mul(f2_pack(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), unit2)};
                float4 k4, l4;
                if constexpr (Q8) k4 = ld_shared_f4(sc + c + e), l4 = ld_shared_f4(sc + BN + c + e);
                if constexpr (!MODS) {
                  t[0] = f2_fma(t[0], f2_pack(k4.x, k4.y), f2_pack(l4.x, l4.y));
                  t[1] = f2_fma(t[1], f2_pack(k4.z, k4.w), f2_pack(l4.z, l4.w));
                } else {
                  if constexpr (Q8) t[0] = f2_mul(t[0], f2_pack(k4.x, k4.y)), t[1] = f2_mul(t[1], f2_pack(k4.z, k4.w));
                  if (p.capped) cap_quad_of(p.cap, t[0], t[1]);
                  float v[4] = {f2_lo(t[0]), f2_hi(t[0]), f2_lo(t[1]), f2_hi(t[1])};
#pragma unroll
                  for (int y = 0; y < 4; ++y) v[y] = fmaf(-slope, far0 - (float)(e + y), v[y]);
                  t[0] = f2_pack(v[0], v[1]), t[1] = f2_pack(v[2], v[3]);
                  if constexpr (Q8) t[0] = f2_add(t[0], f2_pack(l4.x, l4.y)), t[1] = f2_add(t[1], f2_pack(l4.z, l4.w));
                }
                s[e] = __float_as_uint(f2_lo(t[0])), s[e + 1] = __float_as_uint(f2_hi(t[0]));
                s[e + 2] = __float_as_uint(f2_lo(t[1])), s[e + 3] = __float_as_uint(f2_hi(t[1]));
              }
              if (some_hidden) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (e < from || e >= to) s[e] = __float_as_uint(NEG_INF);
              }
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                top[0] = fmax3(top[0], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                top[1] = fmax3(top[1], __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
              }
              tmem_st32(tS + c, s);
            }
            tmem_wait_st();
            mt = fmaxf(top[0], top[1]);
            refer();
            const uint64_t nbase2 = f2_pack(-base, -base);
            uint64_t rs[2] = {0ull, 0ull};
#pragma unroll 1
            for (int c = 0; c < BN; c += 32) {
              uint32_t s[32], pk[16];
              tmem_ld32(tS + c, s);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const uint64_t x0 = f2_add(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), nbase2);
                const uint64_t x1 = f2_add(f2_pack(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), nbase2);
                const float e0 = ex2(f2_lo(x0)), e1 = ex2(f2_hi(x0)), e2 = ex2(f2_lo(x1)), e3 = ex2(f2_hi(x1));
                if constexpr (Q8) {
                  const float4 i4 = ld_shared_f4(sc + 2 * BN + c + e);
                  rs[0] = f2_fma(f2_pack(e0, e1), f2_pack(i4.x, i4.y), rs[0]);
                  rs[1] = f2_fma(f2_pack(e2, e3), f2_pack(i4.z, i4.w), rs[1]);
                } else {
                  rs[0] = f2_add(rs[0], f2_pack(e0, e1));
                  rs[1] = f2_add(rs[1], f2_pack(e2, e3));
                }
                pk[e / 2] = Q8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
                pk[e / 2 + 1] = Q8 ? pack_f16x2(e2, e3) : pack_bf16x2(e2, e3);
              }
              tmem_st16(tS + c / 2, pk);  // (over columns that have been read)
            }
            const uint64_t rs2 = f2_add(rs[0], rs[1]);
            sum = f2_lo(rs2) + f2_hi(rs2);
          } else {
            uint32_t sr[BN];
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
            tmem_wait_ld();
            // Of the columns only those from `from` on and before `lim` count.
            const int from = WINDOW ? pos + lim - p.window + 1 : 0;
            const bool some_hidden = __any_sync(~0u, from > 0 || lim < BN);
            auto hide = [&](uint32_t with) {
#pragma unroll
              for (int c = 0; c < BN; ++c)
                if (c < from || c >= lim) sr[c] = with;
            };
            if constexpr (MODS) {
              const uint64_t unit2 = f2_pack(unit, unit), nslope2 = f2_pack(-slope, -slope);
              const uint64_t far2 = f2_pack((float)(pos + lim), (float)(pos + lim));  // of column 0
#pragma unroll
              for (int c = 0; c < BN; c += 4) {
                uint64_t a = f2_mul(f2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), unit2);
                uint64_t b = f2_mul(f2_pack(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3])), unit2);
                a = f2_fma(nslope2, f2_add(far2, f2_pack((float)-c, (float)(-c - 1))), a);
                b = f2_fma(nslope2, f2_add(far2, f2_pack((float)(-c - 2), (float)(-c - 3))), b);
                sr[c] = __float_as_uint(f2_lo(a)), sr[c + 1] = __float_as_uint(f2_hi(a));
                sr[c + 2] = __float_as_uint(f2_lo(b)), sr[c + 3] = __float_as_uint(f2_hi(b));
              }
            }
            if (some_hidden) hide(__float_as_uint(NEG_INF));
            const float sl = MODS ? 1.f : unit;  // what brings sr to log2 units
            float pm[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) pm[k] = __uint_as_float(sr[k]);
#pragma unroll
            for (int c = 8; c + 16 <= BN; c += 16)
#pragma unroll
              for (int k = 0; k < 8; ++k) pm[k] = fmax3(pm[k], __uint_as_float(sr[c + k]), __uint_as_float(sr[c + 8 + k]));
#pragma unroll
            for (int k = 0; k < 8; ++k) pm[k] = fmaxf(pm[k], __uint_as_float(sr[BN - 8 + k]));
            mt = fmax3(fmax3(pm[0], pm[1], pm[2]), fmax3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7])) * sl;
            refer();
            const uint64_t sl2 = f2_pack(sl, sl), nbase2 = f2_pack(-base, -base);
            uint64_t rs[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint64_t xv = f2_fma(
                    f2_pack(__uint_as_float(sr[32 * c + 2 * e]), __uint_as_float(sr[32 * c + 2 * e + 1])), sl2, nbase2);
                const float e0 = ex2(f2_lo(xv)), e1 = ex2(f2_hi(xv));
                rs[e & 3] = f2_add(rs[e & 3], f2_pack(e0, e1));
                pk[e] = pack_bf16x2(e0, e1);
              }
              tmem_st16(tS + 16 * c, pk);
            }
            const uint64_t rs2 = f2_add(f2_add(rs[0], rs[1]), f2_add(rs[2], rs[3]));
            sum = f2_lo(rs2) + f2_hi(rs2);
          }
          // O_X is idle here: the P.V of tile j - 1 completed before S_X(j) did.
          const float alpha = m_new == m_ref ? 1.f : m_ref == NEG_INF ? 0.f : ex2(m_ref - m_new);
          l = l * alpha + sum;
          if (warp_rescale) {
            const float a = rescale ? alpha : 1.f;
#pragma unroll 1
            for (int c = 0; c < DV / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
              tmem_st32(tO + c * 32, o);
            }
          }
          m_ref = m_new;
          tmem_wait_st();
          tc_fence_before();
          if (there) mbar_arrive(&p_full[x]);
          lim -= step * BN;
        }
        if (ok && tiles > 0) ok = agree(mbar_wait_for(&o_done[x], no++ & 1, abort_flag));
        if (CAREFUL && ok) ok = agree(mbar_wait_for(&found_full[items & 1], (items >> 1) & 1, abort_flag));
        if (ok) {
          tc_fence_after();
          [[maybe_unused]] int last_hidden = INT_MAX;
          [[maybe_unused]] const int* found = found_of(items);
          [[maybe_unused]] const bool some_found = CAREFUL && found[DV] > 0;
          if (some_found) {
            const Cursor it = *walk;
            const fa::CacheRow w = fa::cache_row(p, it.n, first_row(it) + (two_tiles(it) ? x * BM : 0) + r);
            last_hidden = it.n.keys + fa::cache_length(p, w.b) - p.T + w.t - p.window;
          }
          const bool some = s_row[threadIdx.x - 128] != 0, none = s_row[threadIdx.x - 128] == 2 || tiles <= 0;
          const long long at = (((long long)walk->item + share.cta) * walk->bundle + share.tile) * fa::kPrefixRows + x * BM + r;
          if (some) *reinterpret_cast<float2*>(p.parts.ml + at * 2) = none ? make_float2(NEG_INF, 0.f) : make_float2(m_ref, l);
          // 32 columns at a time through this warp's share of Q_X, which is free now, so that a
          // row's 128 bytes leave together.
          uint8_t* stage = smem + x * C::Q_BYTES + quad * 4096;
          const unsigned valid = __ballot_sync(~0u, some);
          const long long first = at - lane;  // the warp's first row
#pragma unroll 1
          for (int c = 0; c < DV / 32; ++c) {
            uint32_t o[32];
            if (tiles > 0) {
              tmem_ld32(tO + c * 32, o);
              tmem_wait_ld();
            }
            if (kLooks && tiles > 0) {
              uint64_t none2 = 0ull;  // 0 times each: 0, or NaN
#pragma unroll
              for (int k = 0; k < 32; k += 2)
                none2 = f2_fma(f2_pack(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), 0ull, none2);
              if (f2_lo(none2) + f2_hi(none2) != 0.f && s_row[threadIdx.x - 128] == 1) *not_finite = 1;
            }
            if (some_found) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (found[c * 32 + k] > last_hidden) o[k] = 0x7fffffffu;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                  none ? make_uint4(0, 0, 0, 0) : make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int row = k * 4 + lane / 8;
              const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
              if ((valid >> row) & 1u)
                *reinterpret_cast<uint4*>(p.parts.part + (first + row) * DV + c * 32 + (lane & 7) * 4) = v;
            }
            __syncwarp();
          }
          tc_fence_before();  // (the next item's first P.V into O_X follows this warpgroup's next P)
          if (CAREFUL) mbar_arrive(&found_free[items++ & 1]);
        }
      }
      units += 2 * (walk->end(p, share.end) - walk->c);
      __syncwarp();
      if (lane == 0) walk->next(p);
      __syncwarp();
    }
  }
  __syncwarp();  // (the MMA thread and the rest of its warp)
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicExch(p.status, DEV_TIMEOUT);
  // (Not before the deallocation, which warp 0 does as a whole: thread 0 would come to it apart.)
  if (kLooks && threadIdx.x == 0) p.look[blockIdx.x] = *not_finite;
}

template <int D, int DV, bool Q8, int MODS, bool WINDOW, bool CAREFUL>
cudaError_t launch_mods(const CacheParams& p, int grid, cudaStream_t stream) {
  using C = PrefixCfg<D, DV, Q8>;
  auto kernel = fa_cache_prefix_kernel<D, DV, Q8, MODS, WINDOW, CAREFUL>;
  cudaError_t e = fa::allow_dynamic_smem(reinterpret_cast<const void*>(kernel), C::SMEM);
  if (e != cudaSuccess) return e;
  // The register split only balances if every thread was launched with kRegsLaunch.
  cudaFuncAttributes a;
  e = cudaFuncGetAttributes(&a, kernel);
  if (e != cudaSuccess) return e;
  if (a.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
  CUtensorMap mk = {}, mv = {};
  const int page = 1 << p.page_log2;
  const long long heads = (long long)p.pages * p.Hkv;
  if (!Q8 && (!fa::encode_pages_bf16(&mk, p.K, D, page, heads, page < BN ? page : BN) ||
              !fa::encode_pages_bf16(&mv, p.V, DV, page, heads, page < BN ? page : BN)))
    return cudaErrorInvalidValue;
  if (CAREFUL) return fa::launch_next(kernel, dim3((unsigned)grid), kThreads, C::SMEM, stream, p, mk, mv);
  kernel<<<grid, kThreads, C::SMEM, stream>>>(p, mk, mv);
  return cudaGetLastError();
}

template <int D, int DV, bool Q8, bool WINDOW, bool CAREFUL>
cudaError_t launch_dims(const CacheParams& p, int grid, cudaStream_t stream) {
  constexpr int kLine = Q8 ? kCapped : kLines;
  if (p.capped) return launch_mods<D, DV, Q8, kCapped, WINDOW, CAREFUL>(p, grid, stream);
  if (WINDOW || p.slopes) return launch_mods<D, DV, Q8, kLine, WINDOW, CAREFUL>(p, grid, stream);
  return launch_mods<D, DV, Q8, WINDOW ? kLine : kUnmodified, WINDOW, CAREFUL>(p, grid, stream);
}

// WINDOW: p.window is not 0.
template <bool Q8, bool WINDOW, bool CAREFUL>
cudaError_t launch_prefix(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream) {
  if (d == 64)
    return dv == 64 ? launch_dims<64, 64, Q8, WINDOW, CAREFUL>(p, grid, stream) : launch_dims<64, 128, Q8, WINDOW, CAREFUL>(p, grid, stream);
  return dv == 64 ? launch_dims<128, 64, Q8, WINDOW, CAREFUL>(p, grid, stream) : launch_dims<128, 128, Q8, WINDOW, CAREFUL>(p, grid, stream);
}

}  // namespace
