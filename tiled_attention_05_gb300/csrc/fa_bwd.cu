// Backward pass: the preprocess and cast kernels, the plain instances of the
// main kernel (fa_bwd_kernel.cuh) and the launcher that picks an instance (the
// score-modified ones are compiled in fa_scored_bwd_*.cu).
#include "fa_bwd_kernel.cuh"

namespace {

// D = rowsum(dO * O) and L2 = L * log2(e) per padded query row (padding rows:
// D = 0, L2 = +inf); zeroes the row of the fp32 dQ accumulator (and the main
// kernel's split-item counters).  HD: columns
// of the accumulator (d); HDV: columns of O and dO (dv).  A row is HDV / 8
// lanes with 16 bytes of O and of dO each; a warp takes two groups of
// 32 / (HDV / 8) rows per step, so that every lane has four 16-byte loads in
// flight (the kernel is short and bound by memory latency as much as by
// bandwidth).
template <int HD, int HDV>
__global__ void __launch_bounds__(256) fa_bwd_pre(const uint16_t* __restrict__ O, const uint16_t* __restrict__ dO,
                                                  const float* __restrict__ L, float* __restrict__ lse2,
                                                  float* __restrict__ delta, float* __restrict__ dq_acc,
                                                  unsigned int* __restrict__ split_counters, int n_counters,
                                                  long long rows_pad, int Tq, long long Tq_pad) {
  grid_next();
  grid_previous();
  if (blockIdx.x == 0)
    for (int c = threadIdx.x; c < n_counters; c += blockDim.x) split_counters[c] = 0u;
  constexpr int LPR = HDV / 8;   // lanes per row
  constexpr int RPG = 32 / LPR;  // rows per group
  constexpr int UNR = 2;         // groups per warp step
  constexpr int ZF4 = HD / (4 * LPR);  // float4 of the accumulator row each lane zeroes
  const int lane = threadIdx.x & 31, sub = lane / LPR, part = lane - sub * LPR;
  const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
  const long long wid = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  for (long long base = wid * (RPG * UNR); base < rows_pad; base += warps * (RPG * UNR)) {
    uint4 a[UNR], g[UNR];
    long long row[UNR], src_row[UNR];
    bool real[UNR];
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      row[u] = base + u * RPG + sub;
      const long long bh = row[u] / Tq_pad;
      const long long q = row[u] - bh * Tq_pad;
      real[u] = row[u] < rows_pad && q < Tq;
      src_row[u] = bh * Tq + q;
      a[u] = g[u] = make_uint4(0u, 0u, 0u, 0u);
      if (real[u]) {
        a[u] = *reinterpret_cast<const uint4*>(O + src_row[u] * HDV + part * 8);
        g[u] = *reinterpret_cast<const uint4*>(dO + src_row[u] * HDV + part * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      const uint32_t aw[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, gw[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dot += __uint_as_float(aw[e] << 16) * __uint_as_float(gw[e] << 16);
        dot += __uint_as_float(aw[e] & 0xffff0000u) * __uint_as_float(gw[e] & 0xffff0000u);
      }
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
      if (row[u] < rows_pad) {
        if (part == 0) {
          delta[row[u]] = dot;
          // a row that saw no key (L = -inf) is treated like padding
          const float l = real[u] ? L[src_row[u]] : -__int_as_float(0x7f800000);
          lse2[row[u]] = l == -__int_as_float(0x7f800000) ? -l : l * 1.4426950408889634f;
        }
        float4* acc = reinterpret_cast<float4*>(dq_acc + row[u] * HD) + part * ZF4;
#pragma unroll
        for (int z = 0; z < ZF4; ++z) acc[z] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
  }
}

// dQ = bf16(scale * accumulator).  A row is HD / 8 lanes with 8 fp32 each;
// a warp takes two groups of 32 / (HD / 8) rows per step (four 16-byte loads
// in flight per lane).
template <int HD>
__global__ void __launch_bounds__(256) fa_dq_cast(const float* __restrict__ dq_acc, uint16_t* __restrict__ dQ,
                                                  long long q_rows, int Tq, long long Tq_pad, float scale) {
  grid_next();
  grid_previous();
  constexpr int LPR = HD / 8;
  constexpr int RPG = 32 / LPR;
  constexpr int UNR = 2;
  const int lane = threadIdx.x & 31, sub = lane / LPR, part = lane - sub * LPR;
  const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
  const long long wid = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  for (long long base = wid * (RPG * UNR); base < q_rows; base += warps * (RPG * UNR)) {
    float4 x[UNR], y[UNR];
    long long row[UNR];
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      row[u] = base + u * RPG + sub;
      x[u] = y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row[u] < q_rows) {
        const long long bh = row[u] / Tq;
        const float* src = dq_acc + (bh * Tq_pad + (row[u] - bh * Tq)) * HD + part * 8;
        x[u] = *reinterpret_cast<const float4*>(src);
        y[u] = *reinterpret_cast<const float4*>(src + 4);
      }
    }
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      if (row[u] >= q_rows) continue;
      uint4 o;
      o.x = pack_bf16x2(x[u].x * scale, x[u].y * scale);
      o.y = pack_bf16x2(x[u].z * scale, x[u].w * scale);
      o.z = pack_bf16x2(y[u].x * scale, y[u].y * scale);
      o.w = pack_bf16x2(y[u].z * scale, y[u].w * scale);
      *reinterpret_cast<uint4*>(dQ + row[u] * HD + part * 8) = o;
    }
  }
}

__global__ void fa_zero_words(uint32_t* p, size_t n) {
  for (size_t t = blockIdx.x * (size_t)blockDim.x + threadIdx.x; t < n; t += (size_t)gridDim.x * blockDim.x) p[t] = 0u;
}

template <int HD, int HDV>
cudaError_t launch_main_dims(const fa::Problem& pr, const CUtensorMap* maps, const BwdParams& bp,
                             cudaStream_t stream) {
  if (!pr.causal) return launch_main_t<HD, HDV, false, false, fa::kPlain>(pr, maps, bp, stream);
  if (pr.window) return launch_main_t<HD, HDV, true, true, fa::kPlain>(pr, maps, bp, stream);
  return launch_main_t<HD, HDV, true, false, fa::kPlain>(pr, maps, bp, stream);
}

// Groups per super-batch of fa_bwd_main's grid order: the smallest divisor of
// the group count whose super-batch holds at least 1.5 CTAs per SM, so that
// one super-batch fills the GPU with a heaviest-first queue of its own while
// few groups' data is live in L2 (with a plan: see planned_super_batch_groups).
// 0 if the SM count cannot be read.
int backward_super_batch(int n_groups, int kv_tiles, bool planned) {
  const int sms = fa::sm_count();
  if (sms <= 0) return 0;
  return planned ? fa::planned_super_batch_groups(n_groups, kv_tiles, sms) : fa::super_batch_groups(n_groups, kv_tiles, sms);
}

inline int grid_for(long long work, int per_block) {
  long long g = (work + per_block - 1) / per_block;
  if (g > 152LL * 32) g = 152LL * 32;
  return (int)(g < 1 ? 1 : g);
}

}  // namespace

namespace fa {

BwdWorkspace backward_workspace_layout(const Problem& p, long long slots, int items) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t rows = (size_t)p.B * p.Hq * (size_t)p.Tq_pad();
  BwdWorkspace w;
  w.dq_acc = 0;
  w.lse2 = up(w.dq_acc + rows * p.d * sizeof(float));
  w.delta = up(w.lse2 + rows * sizeof(float));
  w.part = up(w.delta + rows * sizeof(float));
  w.total_min = w.part;
  // Items have equal work without a causal mask: then a short last round may
  // be split (up to kMaxSplitItems items).  (With a window the last key
  // tiles of each head are lighter, and splitting did not pay.)
  const long long n_items = (long long)p.B * p.Hkv * p.kv_tiles();
  w.split_cap = !p.causal ? (int)(n_items < kMaxSplitItems ? n_items : kMaxSplitItems) : 0;
  if (slots >= 0) w.split_cap = items;
  if (slots < 0) slots = 2LL * w.split_cap;
  w.counters = up(w.part + (size_t)slots * kTile * (p.d + p.dv) * sizeof(float));
  w.total = up(w.counters + (size_t)w.split_cap * sizeof(unsigned int));
  return w;
}

// Items of the backward main kernel run as two halves (each half walks half
// of the item's query tiles and the halves' dK / dV are added): the last
// n_items mod sms items, where items have equal work and that last round
// fills at most half of the SMs, so its halves run on twice as many SMs.
int backward_split_items(const Problem& p, int split_cap) {
  int dev = 0, sms = 0;
  if (split_cap <= 0 || cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    return 0;
  const long long n_items = (long long)p.B * p.Hkv * p.kv_tiles();
  const long long r = n_items % sms;
  return (r > 0 && 2 * r <= sms && r <= split_cap) ? (int)r : 0;
}

cudaError_t launch_backward(const Problem& pr, const ScoreMods& mods, const void* Q, const void* K, const void* V,
                            const void* O, const void* dO, const float* L, void* dQ, void* dK, void* dV, void* workspace,
                            size_t workspace_bytes, int stages, cudaStream_t stream, int* launches) {
  const long long q_rows = (long long)pr.B * pr.Hq * pr.Tq;
  const long long k_rows = (long long)pr.B * pr.Hkv * pr.Tk;
  if (q_rows == 0 && k_rows == 0) return cudaSuccess;
  if (q_rows == 0 || pr.Tk == 0) {
    if (!(stages & FA_BWD_MAIN)) return cudaSuccess;
    // No query rows: dK = dV = 0.  No keys: dQ = 0.
    if (k_rows) {
      fa_zero_words<<<grid_for(k_rows * pr.d / 2, 256), 256, 0, stream>>>(static_cast<uint32_t*>(dK),
                                                                         (size_t)k_rows * pr.d / 2);
      fa_zero_words<<<grid_for(k_rows * pr.dv / 2, 256), 256, 0, stream>>>(static_cast<uint32_t*>(dV),
                                                                          (size_t)k_rows * pr.dv / 2);
      *launches += 2;
    }
    if (q_rows) {
      fa_zero_words<<<grid_for(q_rows * pr.d / 2, 256), 256, 0, stream>>>(static_cast<uint32_t*>(dQ),
                                                                         (size_t)q_rows * pr.d / 2);
      *launches += 1;
    }
    return cudaGetLastError();
  }
  // (modified scores: unequal items in parts where there are few, else the plain rule)
  const ScoredSplit parts = mods.any() ? scored_split(pr, sm_count()) : ScoredSplit{0, 1};
  const BwdWorkspace w = parts.items ? backward_workspace_layout(pr, (long long)parts.items * parts.parts, parts.items)
                                     : backward_workspace_layout(pr);
  // the split items' area is used only where the caller's workspace holds it
  const int split_cap = workspace_bytes >= w.total ? w.split_cap : 0;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* dq_acc = reinterpret_cast<float*>(ws + w.dq_acc);
  float* lse2 = reinterpret_cast<float*>(ws + w.lse2);
  float* delta = reinterpret_cast<float*>(ws + w.delta);
  float* part = reinterpret_cast<float*>(ws + w.part);
  unsigned int* split_counters = reinterpret_cast<unsigned int*>(ws + w.counters);
  const long long rows_pad = (long long)pr.B * pr.Hq * pr.Tq_pad();

  cudaError_t e = cudaSuccess;
  // 1. preprocess
  if (stages & FA_BWD_PRE) {
  auto pre = pr.d == 64 ? (pr.dv == 64 ? fa_bwd_pre<64, 64> : fa_bwd_pre<64, 128>)
                        : (pr.dv == 64 ? fa_bwd_pre<128, 64> : fa_bwd_pre<128, 128>);
  e = launch_next(pre, grid_for(rows_pad, 8 * 2 * (32 / (pr.dv / 8))), 256, 0, stream, static_cast<const uint16_t*>(O),
                  static_cast<const uint16_t*>(dO), L, lse2, delta, dq_acc, split_counters, split_cap, rows_pad, pr.Tq,
                  pr.Tq_pad());
  if (e != cudaSuccess) return e;
  ++*launches;
  }

  // 2. main
  if (stages & FA_BWD_MAIN) {
  CUtensorMap maps[7];
  if (!encode_rows_bf16(&maps[0], Q, pr.d, pr.Tq, (long long)pr.B * pr.Hq) ||
      !encode_rows_bf16(&maps[1], K, pr.d, pr.Tk, (long long)pr.B * pr.Hkv) ||
      !encode_rows_bf16(&maps[2], V, pr.dv, pr.Tk, (long long)pr.B * pr.Hkv) ||
      !encode_rows_bf16(&maps[3], dO, pr.dv, pr.Tq, (long long)pr.B * pr.Hq) ||
      !encode_rows_bf16(&maps[4], dK, pr.d, pr.Tk, (long long)pr.B * pr.Hkv) ||
      !encode_rows_bf16(&maps[5], dV, pr.dv, pr.Tk, (long long)pr.B * pr.Hkv) ||
      !encode_acc_f32(&maps[6], dq_acc, pr.d, pr.Tq_pad(), (long long)pr.B * pr.Hq, 32))
    return cudaErrorInvalidValue;
  ScoredBwdParams bp;
  bp.lse2 = lse2;
  bp.delta = delta;
  bp.status = device_status_word();
  bp.Hq = pr.Hq;
  bp.Hkv = pr.Hkv;
  bp.G = pr.G();
  bp.Tq = pr.Tq;
  bp.Tk = pr.Tk;
  bp.causal_off = pr.Tk - pr.Tq;
  bp.window = pr.causal ? pr.window : 0;
  bp.q_tiles = pr.q_tiles();
  bp.kv_tiles = pr.kv_tiles();
  // (items in parts: the heaviest of all first)
  bp.sb_groups = parts.items ? pr.B * pr.Hkv : backward_super_batch(pr.B * pr.Hkv, pr.kv_tiles(), mods.plan != nullptr);
  if (bp.sb_groups < 1) return cudaErrorInvalidValue;
  bp.Tq_pad = pr.Tq_pad();
  bp.scale_grad = scale_grad(pr, mods);
  bp.scale_log2 = pr.scale * 1.4426950408889634f;
  bp.test_withhold_do = fa::test_withhold() == fa::kWithholdBwdDO;
  bp.cap = cap_params(mods.softcap, pr.scale);
  bp.slopes = mods.slopes;
  bp.hi_off = row_hi_off(pr);
  bp.lo_off = row_lo_off(pr);
  bp.two_sided = !pr.causal || mods.plan;
  bp.plan = plan_view(pr, mods.plan);
  bp.parts = parts.items ? parts.parts : 2;
  bp.split_first = parts.items != 0;
  bp.n_split = parts.items ? split_cap : mods.plan ? 0 : backward_split_items(pr, split_cap);
  bp.n_whole = (int)((long long)pr.B * pr.Hkv * pr.kv_tiles()) - bp.n_split;
  bp.part = part;
  bp.split_counters = split_counters;
  if (mods.any())
    e = pr.d == 64 ? launch_bwd_scored_64(pr, mods, maps, bp, stream) : launch_bwd_scored_128(pr, mods, maps, bp, stream);
  else if (pr.d == 64)
    e = pr.dv == 64 ? launch_main_dims<64, 64>(pr, maps, bp, stream) : launch_main_dims<64, 128>(pr, maps, bp, stream);
  else
    e = pr.dv == 64 ? launch_main_dims<128, 64>(pr, maps, bp, stream)
                    : launch_main_dims<128, 128>(pr, maps, bp, stream);
  if (e != cudaSuccess) return e;
  ++*launches;
  }

  // 3. dQ cast
  if (!(stages & FA_BWD_CAST)) return cudaSuccess;
  const int rows_per_block = 8 * 2 * (32 / (pr.d / 8));  // 8 warps, two row groups each
  auto cast = pr.d == 64 ? fa_dq_cast<64> : fa_dq_cast<128>;
  e = launch_next(cast, grid_for(q_rows, rows_per_block), 256, 0, stream, dq_acc, static_cast<uint16_t*>(dQ), q_rows, pr.Tq,
                  pr.Tq_pad(), scale_grad(pr, mods));
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace fa
