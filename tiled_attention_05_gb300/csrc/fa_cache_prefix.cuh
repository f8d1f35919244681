// Attention of many rows over one shared prefix (fa_cache_attention): the rows of all
// sequences of a group meet the prefix's keys at once, on the tcgen05 tensor cores.
// What comes out are parts (unnormalised O, reference, sum) that the join adds to those
// of the sequences' own keys.
//
// An item is (group, kv head, up to 256 rows), two tiles of 128; the list of items times
// key tiles of 128 is cut into equal shares, one CTA an SM each.  Roles:
//   warp 0       issues the MMAs of both tiles in turn, S_X(j) = Q_X K_j^T and
//                O_X += P_X(j) V_j, so that the tensor pipe runs one tile's while the
//                softmax works on the other's (the forward's order: those of one
//                thread execute in issue order, so S_X(j + 1) may overwrite P_X(j))
//   warps 1..3   bring K_j and V_j from their pages into the ring's slots, in the 128-byte
//                swizzle that TMA would write: rows lie in pages of 16 and more, some
//                of a tile past the prefix's end, and e4m3 codes become fp16 on the way
//                (16 cp.async of a slot in flight while the one before it is converted)
//   warps 4..11  softmax of tile A and of tile B, a thread a row: scores from TMEM, exp2, P
//                as 16-bit pairs over the scores, O rescaled in TMEM when the maximum grows
//                by more than 2^8; before that the row of Q into shared memory, after
//                it the part to the workspace
// e4m3: as in fa_cache_attn.cuh, codes and weights meet in fp16, the key's scale
// multiplies the score, the value's goes into the exponent.  (Codes could feed the fp8
// pipe as they are, but then the weights would be e4m3 too: a sum of two has a weight's
// 8 bits, and ends at 2^-18 of the largest, which a long flat tail falls below.)
// MODS: cap, slopes and window.
#pragma once
#include <cstdint>
#include <type_traits>

#include "fa_cache_internal.h"
#include "sm103_ptx.cuh"

namespace {

using namespace fa_ptx;
using fa::CacheEntry;
using fa::CacheParams;

constexpr int kThreads = 384, kLoaders = 96;
constexpr int BM = 128, BN = fa::kPrefixKeys;
// Register split, as in the forward: 88 + 2 * 208 = 3 * 168.
constexpr int kRegsLaunch = 168, kRegsLow = 88, kRegsHigh = 208;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: weights stay <= 256

template <int D, int DV, bool Q8>
struct PrefixCfg {
  static constexpr int W = D > DV ? D : DV;
  static constexpr int Q_BYTES = BM * D * 2, SLOT = BN * W * 2;
  static constexpr int RAW = Q8 ? BN * W : 0;  // a slot's codes, in the order of the copying threads
  static constexpr int NRAW = Q8 ? 3 : 0;
  static constexpr int SCALES = Q8 ? 2 * 2 * 3 * BN * 4 : 0;  // [tile][buffer][k_scale, log2 v_scale, 1 / v_scale][key]
  static constexpr int OFF_SLOT = 2 * Q_BYTES;
  static constexpr int ROOM = (226 << 10) - 1024 - OFF_SLOT - NRAW * RAW - SCALES;
  static constexpr int NS = ROOM / SLOT > 6 ? 6 : ROOM / SLOT;
  static constexpr int OFF_RAW = OFF_SLOT + NS * SLOT;
  static constexpr int OFF_SCALES = OFF_RAW + NRAW * RAW;
  static constexpr int OFF_BAR = OFF_SCALES + SCALES;
  static constexpr int SMEM = OFF_BAR + 512;
  // V_j leaves its slot after S_A(j + 1), so a loader must not wait for that before K_{j+1}
  // is handed over: two slots, and as many as copies it has in flight beyond (bf16).
  static_assert(NS >= (Q8 ? 2 : 4) && SMEM <= (226 << 10), "shared memory");
};

// Instruction descriptor, kind::f16 with fp32 D; A and B fp16 or bf16.
__host__ __device__ constexpr uint32_t idesc(bool f16, int M, int N, int b_mn) {
  return f16 ? idesc_bf16(M, N, 0, b_mn) & ~((1u << 7) | (1u << 10)) : idesc_bf16(M, N, 0, b_mn);
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t half2_of(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 c, u;\n\tmov.b32 {c, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float capped(const fa::CapParams& c, float x) {
  const float u = x * x;
  if (u <= c.small2) return x * (c.a[0] + u * (c.a[1] + u * (c.a[2] + u * (c.a[3] + u * c.a[4]))));
  return c.log2c - 2.f * c.log2c * rcp(1.f + ex2(cap_top<true>(c.in * x)));
}

template <int D, int DV, bool Q8, bool MODS>
__global__ void __launch_bounds__(kThreads, 1) fa_cache_prefix_kernel(const CacheParams p) {
  using C = PrefixCfg<D, DV, Q8>;
  using Cursor = fa::CacheCursor<BN, fa::kPrefixRows>;
  constexpr int NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  grid_next();
  grid_previous();
  const bool groups_ok = fa::cache_groups_ok(p);
  const auto share = fa::cache_share<BN, fa::kPrefixRows, kThreads>(p, groups_ok);
  if (share.begin >= share.end) return;

  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [NS] a slot holds its tile
  uint64_t* empty = full + NS;     // [NS]
  uint64_t* q_full = empty + NS;   // [2]
  uint64_t* s_full = q_full + 2;   // [2]
  uint64_t* p_full = s_full + 2;   // [2]
  uint64_t* o_done = p_full + 2;   // [2]
  uint64_t* drain = o_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    *abort_flag = (smem_u32(smem) & 1023u) ? 1 : 0;  // swizzled tiles need 1024 B alignment
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], kLoaders / 32);
      mbar_init(&empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 128);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 128);
      mbar_init(&o_done[x], 1);
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
    const long long left = share.end - it.at;
    return Item{it.c, left < it.n.chunks - it.c ? it.c + (int)left : it.n.chunks};
  };
  auto tile_active = [](const Cursor& it, int x) { return it.n.rows > it.r * fa::kPrefixRows + x * BM; };

  if (warp < 4) {
    setmaxnreg_dec<kRegsLow>();
    if (warp == 0) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0 && run) {
        constexpr uint32_t idS = idesc(Q8, BM, BN, 0), idPV = idesc(Q8, BM, DV, 1);
        const uint32_t q_buf = smem_u32(smem), slots = smem_u32(smem + C::OFF_SLOT);
        int u = 0;  // ring position of the item's first K (K_j at u + 2 j, V_j after it)
        int nq[2] = {0, 0}, np[2] = {0, 0};
        bool ok = true;
        Cursor it = share.start;
        while (ok && it.at < share.end) {
          const Item m = item_of(it);
          const int tiles = m.c1 - m.c0, last_x = tile_active(it, 1) ? 1 : 0;
          auto issue_s = [&](int x, int j) -> bool {
            if (j == 0) {
              if (!mbar_wait(&q_full[x], nq[x] & 1, abort_flag)) return false;
              ++nq[x];
            }
            const int pos = u + 2 * j, s = pos % NS;
            if (x == 0 && !mbar_wait(&full[s], (pos / NS) & 1, abort_flag)) return false;
            tc_fence_after();
            const uint64_t a0 = desc_kmajor(q_buf + x * C::Q_BYTES), b0 = desc_kmajor(slots + s * C::SLOT);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t step = (k >> 2) * (BM * 128) + (k & 3) * 32;
              mma_ss(tmem + x * 128, desc_at(a0, step), desc_at(b0, step), idS, k > 0 ? 1u : 0u);
            }
            mma_commit(&s_full[x]);
            if (x == last_x) mma_commit(&empty[s]);
            return true;
          };
          auto issue_pv = [&](int x, int j) -> bool {
            const int pos = u + 2 * j + 1, s = pos % NS;
            if (!mbar_wait(&p_full[x], np[x] & 1, abort_flag)) return false;
            ++np[x];
            if (x == 0 && !mbar_wait(&full[s], (pos / NS) & 1, abort_flag)) return false;
            tc_fence_after();
            const uint64_t v0 = desc_mnmajor(slots + s * C::SLOT, BN * 128);
#pragma unroll
            for (int k = 0; k < BN / 16; ++k)
              mma_ts(tmem + 256 + x * 128, tmem + x * 128 + k * 8, desc_at(v0, k * 2048), idPV, (j > 0 || k > 0) ? 1u : 0u);
            if (x == last_x) mma_commit(&empty[s]);
            return true;
          };
          for (int x = 0; ok && x <= last_x; ++x) ok = issue_s(x, 0);
          for (int j = 0; ok && j < tiles; ++j)
            for (int x = 0; ok && x <= last_x; ++x) {
              ok = issue_pv(x, j);
              if (!ok) break;
              if (j + 1 < tiles)
                ok = issue_s(x, j + 1);
              else
                mma_commit(&o_done[x]);
            }
          u += 2 * tiles;
          it.advance(p, groups_ok, tiles);
        }
        // Let every MMA issued above finish before TMEM is released.
        mma_commit(drain);
        mbar_wait_bounded(drain, 0);
      }
    } else {
      // ------------------------------------------------------------ loaders
      const int tid = threadIdx.x - 32;
      const uint32_t slots = smem_u32(smem + C::OFF_SLOT), raw = smem_u32(smem + C::OFF_RAW);
      // Pieces of 16 bytes: a row has PK (PV) of them; thread tid takes piece tid % P of
      // rows tid / P + k * (96 / P).
      auto copy = [&](const Cursor& it, int c, bool v, uint32_t dst) {
        const int key0 = (it.n.chunk0 + c) * BN;
        const int* tab = p.p_tables + (long long)it.e * p.p_cols;
        auto go = [&](auto row_bytes) {
          constexpr int B = decltype(row_bytes)::value, P = B / 16, STEP = kLoaders / P;
          const uint8_t* pool = v ? p.V : p.K;
          const int piece = tid % P;
          bool bad = false;
#pragma unroll 4
          for (int k = 0; k < (BN + STEP - 1) / STEP; ++k) {
            const int row = tid / P + k * STEP, key = key0 + row;
            if (row >= BN) break;
            bool ok = key < it.n.keys;
            int id = 0;
            if (ok) {
              id = __ldg(tab + (key >> p.page_log2));
              ok = (unsigned)id < (unsigned)p.pages;
              bad = bad || !ok;
            }
            const long long at = ok ? ((((long long)id * p.Hkv + it.h) << p.page_log2) | (key & page_mask)) * B + piece * 16 : 0;
            const uint32_t to = Q8 ? (uint32_t)(k * kLoaders + tid) * 16
                                   : (piece >> 3) * (BN * 128) + sw128_offset(row, piece & 7);
            cp16(dst + to, pool + at, ok);
          }
          if (bad) fa::cache_bad(p.status);
        };
        if (v)
          go(std::integral_constant<int, DV * (Q8 ? 1 : 2)>{});
        else
          go(std::integral_constant<int, D * (Q8 ? 1 : 2)>{});
      };
      // e4m3: the thread's own pieces, 16 codes each, to fp16 in the slot
      auto convert = [&](bool v, uint32_t src, uint32_t dst) {
        auto go = [&](auto row_bytes) {
          constexpr int P = decltype(row_bytes)::value / 16, STEP = kLoaders / P;
          const int piece = tid % P;
#pragma unroll 4
          for (int k = 0; k < (BN + STEP - 1) / STEP; ++k) {
            const int row = tid / P + k * STEP;
            if (row >= BN) break;
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(src + (k * kLoaders + tid) * 16)
                         : "memory");
            const uint32_t block = dst + (piece >> 2) * (BN * 128);
#pragma unroll
            for (int x = 0; x < 2; ++x)
              st_shared_v4(block + sw128_offset(row, (piece & 3) * 2 + x), half2_of(w[2 * x]), half2_of(w[2 * x] >> 16),
                           half2_of(w[2 * x + 1]), half2_of(w[2 * x + 1] >> 16));
          }
        };
        if (v)
          go(std::integral_constant<int, DV>{});
        else
          go(std::integral_constant<int, D>{});
      };
      // Units K_0, V_0, K_1, ... of all items; `ahead` copies in flight.  Unit u goes to slot
      // u % NS (e4m3: by way of the raw buffer u % NRAW).
      constexpr int AHEAD = 2;
      Cursor ld = share.start;
      Item m = item_of(ld);
      int c = m.c0;
      bool v = false, more = run, ok = run;
      int issued = 0, done = 0;
      uint32_t is_v = 0;  // bit i: unit i (mod 32) is a V
      auto issue = [&]() {  // the next unit, if there is one (a group is committed all the same)
        if (more && ok) {
          if (!Q8 && !mbar_wait(&empty[issued % NS], ((issued / NS) & 1) ^ 1, abort_flag)) ok = false;
          ok = __all_sync(~0u, ok);
          if (ok) {
            copy(ld, c, v, Q8 ? raw + (issued % (C::NRAW + !C::NRAW)) * C::RAW : slots + (issued % NS) * C::SLOT);
            is_v = (is_v & ~(1u << (issued & 31))) | ((uint32_t)v << (issued & 31));
            ++issued;
            v = !v;
            if (!v && ++c == m.c1) {
              ld.advance(p, groups_ok, m.c1 - m.c0);
              more = ld.at < share.end;
              if (more) m = item_of(ld), c = m.c0;
            }
          }
        }
        cp_commit();
      };
      for (int k = 0; k < AHEAD; ++k) issue();
      while (ok && done < issued) {
        issue();
        cp_wait<AHEAD>();  // unit `done` has landed (this thread's pieces of it)
        if (Q8) {
          if (!mbar_wait(&empty[done % NS], ((done / NS) & 1) ^ 1, abort_flag)) ok = false;
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          convert((is_v >> (done & 31)) & 1u, raw + (done % (C::NRAW + !C::NRAW)) * C::RAW, slots + (done % NS) * C::SLOT);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[done % NS]);
        ++done;
      }
      cp_wait<0>();
    }
  } else {
    // ------------------------------------------------------------ softmax of tile x
    setmaxnreg_inc<kRegsHigh>();
    const int x = (warp - 4) >> 2, quad = warp & 3, r = quad * 32 + lane;  // r: row inside the tile == TMEM lane
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_base, tO = tmem + 256 + x * 128 + lane_base;
    const float NEG_INF = -__int_as_float(0x7f800000);
    int ns = 0, no = 0, nb = 0;  // phases waited for; scale buffers written
    int item = share.item;
    bool ok = run;
    // Loads from TMEM are a warp's, and the barrier that hands the scales round is the
    // tile's: those who meet there leave together when one of them gave up.
    auto agree = [&](bool fine) { return Q8 ? named_bar_and(1 + x, 128, fine) : (bool)__all_sync(~0u, fine); };
    Cursor it = share.start;
    while (ok && it.at < share.end) {
      const Item m = item_of(it);
      const int tiles = m.c1 - m.c0;
      if (tile_active(it, x)) {
        const int row = it.r * fa::kPrefixRows + x * BM + r;
        const fa::CacheRow w = fa::cache_row(p, it.n, row);
        const int pos = fa::cache_length(p, w.b) - p.T + w.t;  // among the own keys; negative: padding
        const int head = it.h * p.G + w.g;
        float unit = MODS && p.capped ? 1.f : p.scale_log2;
        const float slope = MODS && p.slopes ? __ldg(p.slopes + head) * 1.4426950408889634f : 0.f;
        const int abs0 = it.n.keys + pos;
        {  // Q's row into shared memory (e4m3: as fp16, its largest value brought to [1, 2))
          const uint4* src = reinterpret_cast<const uint4*>(p.Q + (((long long)w.b * p.Hq + head) * p.T + w.t) * D);
          const uint32_t dst = smem_u32(smem) + x * C::Q_BYTES;
          uint4 q[D / 8];
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < D / 8; ++k) {
            q[k] = w.valid ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
            const uint32_t a[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) top = max(top, max(a[y] & 0x7fffu, (a[y] >> 16) & 0x7fffu));
          }
          const int ex = min(max((int)(top >> 7), 1), 253);
          const float down = __uint_as_float((uint32_t)(254 - ex) << 23);
          if constexpr (Q8) unit *= __uint_as_float((uint32_t)ex << 23);
#pragma unroll
          for (int k = 0; k < D / 8; ++k) {
            uint32_t a[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
            if constexpr (Q8) {
#pragma unroll
              for (int y = 0; y < 4; ++y)
                a[y] = pack_f16x2(__uint_as_float(a[y] << 16) * down, __uint_as_float(a[y] & 0xffff0000u) * down);
            }
            st_shared_v4(dst + (k >> 3) * (BM * 128) + sw128_offset(r, k & 7), a[0], a[1], a[2], a[3]);
          }
          fence_async_smem();
          mbar_arrive(&q_full[x]);
        }
        // The scales of a tile's keys, one key a thread, a tile ahead.
        float ks = 0.f, vs = 0.f;
        auto fetch_scales = [&](int c) {
          const int key = (it.n.chunk0 + c) * BN + r;
          ks = 0.f, vs = 1.f;
          if (key >= it.n.keys) return;
          const int id = __ldg(p.p_tables + (long long)it.e * p.p_cols + (key >> p.page_log2));
          if ((unsigned)id >= (unsigned)p.pages) return;
          const long long at = (((long long)id * p.Hkv + it.h) << p.page_log2) | (key & page_mask);
          ks = __ldg(p.k_scale + at);
          vs = __ldg(p.v_scale + at);
        };
        if constexpr (Q8) fetch_scales(m.c0);
        float m_ref = NEG_INF, l = 0.f;
        for (int j = 0; ok && j < tiles; ++j) {
          const float* sc = nullptr;
          if constexpr (Q8) {
            float* to = reinterpret_cast<float*>(smem + C::OFF_SCALES) + (x * 2 + (nb & 1)) * 3 * BN;
            ++nb;
            const float a = lg2(fmaxf(vs, 0x1p-69f));  // (see fa_cache_attn.cuh)
            to[r] = ks;
            to[BN + r] = vs == vs ? a : vs;
            to[2 * BN + r] = ex2(-a);
            sc = to;
            if (j + 1 < tiles) fetch_scales(m.c0 + j + 1);
          }
          ok = mbar_wait(&s_full[x], ns & 1, abort_flag);
          ok = agree(ok);
          if (!ok) break;
          ++ns;
          tc_fence_after();
          const int kv0 = (it.n.chunk0 + m.c0 + j) * BN;
          uint32_t sr[BN];
#pragma unroll
          for (int c = 0; c < BN / 32; ++c) tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
          tmem_wait_ld();
          if constexpr (Q8 || MODS) {
#pragma unroll
            for (int c = 0; c < BN; c += 4) {
              float t[4];
              float4 k4 = make_float4(1.f, 1.f, 1.f, 1.f), l4 = make_float4(0.f, 0.f, 0.f, 0.f);
              if constexpr (Q8) k4 = ld_shared_f4(sc + c), l4 = ld_shared_f4(sc + BN + c);
              const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, ll[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                t[y] = __uint_as_float(sr[c + y]) * unit;
                if constexpr (!MODS) {
                  t[y] = fmaf(t[y], kk[y], ll[y]);
                } else {
                  if constexpr (Q8) t[y] *= kk[y];
                  if (p.capped) t[y] = capped(p.cap, t[y]);
                  const int far = abs0 - (kv0 + c + y);
                  t[y] -= slope * (float)far;
                  if (p.window && far >= p.window) t[y] = NEG_INF;
                  if constexpr (Q8) t[y] += ll[y];
                }
                sr[c + y] = __float_as_uint(t[y]);
              }
            }
          }
          if (kv0 + BN > it.n.keys) {
#pragma unroll
            for (int c = 0; c < BN; ++c)
              if (kv0 + c >= it.n.keys) sr[c] = __float_as_uint(NEG_INF);
          }
          float pm[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) pm[k] = __uint_as_float(sr[k]);
#pragma unroll
          for (int c = 8; c + 16 <= BN; c += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) pm[k] = fmax3(pm[k], __uint_as_float(sr[c + k]), __uint_as_float(sr[c + 8 + k]));
#pragma unroll
          for (int k = 0; k < 8; ++k) pm[k] = fmaxf(pm[k], __uint_as_float(sr[BN - 8 + k]));
          const float sl = Q8 || MODS ? 1.f : unit;  // what brings sr to log2 units
          const float mt = fmax3(fmax3(pm[0], pm[1], pm[2]), fmax3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7])) * sl;
          float m_new = m_ref;
          if (mt > m_ref + kRescaleThreshold) m_new = mt;  // also taken when m_ref == -inf
          const bool rescale = j > 0 && m_new != m_ref && m_ref != NEG_INF;
          const bool warp_rescale = __any_sync(~0u, rescale);
          const float base = m_new == NEG_INF ? 0.f : m_new;
          const uint64_t sl2 = f2_pack(sl, sl), nbase2 = f2_pack(-base, -base);
          uint64_t rs[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int c = 0; c < BN / 32; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float4 i4 = make_float4(1.f, 1.f, 1.f, 1.f);
              if constexpr (Q8) i4 = ld_shared_f4(sc + 2 * BN + 32 * c + 2 * e);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint64_t s2 = f2_pack(__uint_as_float(sr[32 * c + 2 * e + 2 * y]), __uint_as_float(sr[32 * c + 2 * e + 2 * y + 1]));
                const uint64_t xv = Q8 || MODS ? f2_add(s2, nbase2) : f2_fma(s2, sl2, nbase2);
                const float e0 = ex2(f2_lo(xv)), e1 = ex2(f2_hi(xv));
                if constexpr (Q8)
                  rs[e / 2 & 3] = f2_fma(f2_pack(e0, e1), y ? f2_pack(i4.z, i4.w) : f2_pack(i4.x, i4.y), rs[e / 2 & 3]);
                else
                  rs[e / 2 & 3] = f2_add(rs[e / 2 & 3], f2_pack(e0, e1));
                pk[e + y] = Q8 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
              }
            }
            tmem_st16(tS + 16 * c, pk);
          }
          const uint64_t rs2 = f2_add(f2_add(rs[0], rs[1]), f2_add(rs[2], rs[3]));
          // O_X is idle here: the P.V of tile j - 1 completed before S_X(j) did.
          const float alpha = m_new == m_ref ? 1.f : m_ref == NEG_INF ? 0.f : ex2(m_ref - m_new);
          l = l * alpha + f2_lo(rs2) + f2_hi(rs2);
          if (warp_rescale) {
            const float a = rescale ? alpha : 1.f;
#pragma unroll
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
          mbar_arrive(&p_full[x]);
        }
        if (ok) ok = agree(mbar_wait(&o_done[x], no & 1, abort_flag));
        ++no;
        if (ok) {
          tc_fence_after();
          // A padding row's part is none.
          const bool none = pos < 0;
          const long long at = ((long long)item + blockIdx.x) * fa::kPrefixRows + x * BM + r;
          if (w.valid) *reinterpret_cast<float2*>(p.parts.ml + at * 2) = none ? make_float2(NEG_INF, 0.f) : make_float2(m_ref, l);
          float4* out = reinterpret_cast<float4*>(p.parts.part + at * DV);
#pragma unroll
          for (int c = 0; c < DV / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_wait_ld();
            if (w.valid) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                out[c * 8 + k] = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                                      : make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                                    __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
            }
          }
          tc_fence_before();  // (the next item's first P.V into O_X follows this warpgroup's next P)
        }
      }
      item += m.c1 == it.n.chunks;
      const int old = it.e;
      it.advance(p, groups_ok, tiles);
      for (int e = old + 1; e < it.e && e < p.entries; ++e) item += p.Hkv * fa::cache_entry<BN>(p, e, groups_ok).tiles(fa::kPrefixRows);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicExch(p.status, DEV_TIMEOUT);
}

template <int D, int DV, bool Q8, bool MODS>
cudaError_t launch_mods(const CacheParams& p, int grid, cudaStream_t stream) {
  using C = PrefixCfg<D, DV, Q8>;
  auto kernel = fa_cache_prefix_kernel<D, DV, Q8, MODS>;
  cudaError_t e = fa::allow_dynamic_smem(reinterpret_cast<const void*>(kernel), C::SMEM);
  if (e != cudaSuccess) return e;
  // The register split only balances if every thread was launched with kRegsLaunch.
  cudaFuncAttributes a;
  e = cudaFuncGetAttributes(&a, kernel);
  if (e != cudaSuccess) return e;
  if (a.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
  return fa::launch_next(kernel, dim3((unsigned)grid), kThreads, C::SMEM, stream, p);
}

template <int D, int DV, bool Q8>
cudaError_t launch_dims(const CacheParams& p, int grid, cudaStream_t stream) {
  return p.capped || p.slopes || p.window ? launch_mods<D, DV, Q8, true>(p, grid, stream)
                                          : launch_mods<D, DV, Q8, false>(p, grid, stream);
}

template <bool Q8>
cudaError_t launch_prefix(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream) {
  if (d == 64) return dv == 64 ? launch_dims<64, 64, Q8>(p, grid, stream) : launch_dims<64, 128, Q8>(p, grid, stream);
  return dv == 64 ? launch_dims<128, 64, Q8>(p, grid, stream) : launch_dims<128, 128, Q8>(p, grid, stream);
}

}  // namespace
