// The key/value cache: writing new rows into its pages, reading them back, the join of
// the attention's parts, and the C ABI of all three (fa_cache_* in include/fa.h).
//
// Write.  A row x of d values becomes e4m3 codes and one scale: with a = max |x| (2^-60
// at least), code = e4m3(x * (448 / a)), scale = a * (1 / 448): two fp32 roundings
// before the one to e4m3.  A row with a NaN or an infinity gets codes 0 and scale NaN,
// so that its bytes are finite wherever its weight is 0.  bf16 caches take the row as
// it is.  Read back: bf16(code * scale).
//
// Mapping.  Both are bound by HBM: each byte is read once and written once.  A thread
// owns some channels of a position's key and value, the lanes of a row agree on its maximum
// by shuffles, and a thread has several positions in flight.
#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "fa_cache_internal.h"
#include "sm103_ptx.cuh"

using namespace fa_ptx;
using fa::CacheParams;
using fa::CacheSlots;
using fa::kCacheRows;

namespace {

constexpr int kThreads = 128;
// Positions in flight per thread.  Blocks of 256 and more in flight were slower (write of
// T 8192, B 2, 8 heads of 128: 17.5, 19.3 and 22.9 us with 1, 2 and 4).
template <bool WRITE, bool Q8>
constexpr int kUnroll = WRITE && Q8 ? 1 : 2;
constexpr float kE4m3Max = 448.f, kLeast = 0x1p-60f;

struct PageParams {
  const int *tables, *lengths;  // (write: the counts, or NULL)
  const int* starts;            // write
  int B, H, T, cols, pages, page_log2;
  fa::Divide by_inner, by_outer;  // the rows' order: by T and H (token by token), or H and T (write, `heads_first`)
  int heads_first;
  int* status;
  struct Side {  // K or V
    uint8_t* pool;
    float* scale;
    uint16_t* rows;          // the new rows, or the result
    long long sb, sh, st;    // their strides (elements)
  } side[2];
  int units;  // B * H * T
};

// Row of the pools for position `pos` of sequence b and head h; -1 where the table has
// none.  (T = 2^31 positions do not meet: the capacity is below 2^30.)
__device__ __forceinline__ long long pool_row(const PageParams& p, int b, int h, long long pos) {
  const long long col = pos >> p.page_log2;
  int id = -1;
  if (pos >= 0 && col < p.cols) id = __ldg(p.tables + (long long)b * p.cols + col);
  if ((unsigned)id >= (unsigned)p.pages) {
    fa::cache_bad(p.status);
    return -1;
  }
  return (((long long)id * p.H + h) << p.page_log2) | (pos & ((1 << p.page_log2) - 1));
}

struct Unit {
  int b, h, t;
};
__device__ __forceinline__ Unit unit_of(const PageParams& p, int n) {
  const int outer = p.by_inner(n), inner = n - outer * (int)p.by_inner.by;
  Unit u;
  u.b = p.by_outer(outer);
  const int middle = outer - u.b * (int)p.by_outer.by;
  u.h = p.heads_first ? inner : middle;
  u.t = p.heads_first ? middle : inner;
  return u;
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\t"
      "mov.b32 %0, {x, y};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The lanes of a row hold some channels each, for the same position's row of both K and V:
// where it goes is worked out once for the two.  A lane that quantises has 16 (its
// instructions are the bound then: a thread for each of K and V 29 us, 8 channels 21, 16
// channels 17.5, of T 8192 as above); one that reads back has 8, since its two halves of 32 bytes
// would leave by two stores (17.7 us, 16 channels 20.8).  LANES: of this row; the wider
// of the two decides the group's size.
template <bool Q8>
constexpr int kChannels = Q8 ? 16 : 8;  // write
template <bool Q8>
struct Piece {
  uint4 x[Q8 ? 2 : 1];
};

template <int LANES, bool Q8>
__device__ __forceinline__ void write_row(const PageParams::Side& s, const Piece<Q8>& piece, long long to, int lane) {
  if constexpr (Q8) {
    const uint32_t w[8] = {piece.x[0].x, piece.x[0].y, piece.x[0].z, piece.x[0].w, piece.x[1].x, piece.x[1].y, piece.x[1].z, piece.x[1].w};
    uint32_t two = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) two = __vmaxu2(two, w[k] & 0x7fff7fffu);
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) two = __vmaxu2(two, __shfl_xor_sync(~0u, two, o));
    const uint32_t top = max(two & 0xffffu, two >> 16);
    const bool finite = top < 0x7f80u;
    const float a = fmaxf(__uint_as_float(top << 16), kLeast);
    const float f = finite ? __fdiv_rn(kE4m3Max, a) : 0.f;
    const uint64_t f2 = f2_pack(f, f);
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t u = f2_mul(f2_pack(bf_lo(w[2 * k]), bf_hi(w[2 * k])), f2), v = f2_mul(f2_pack(bf_lo(w[2 * k + 1]), bf_hi(w[2 * k + 1])), f2);
      c[k] = finite ? codes4(f2_lo(u), f2_hi(u), f2_lo(v), f2_hi(v)) : 0u;
    }
    if (to < 0 || lane >= LANES) return;
    *reinterpret_cast<uint4*>(s.pool + to * (LANES * 16) + lane * 16) = make_uint4(c[0], c[1], c[2], c[3]);
    if (lane == 0) s.scale[to] = finite ? a * (1.f / kE4m3Max) : __uint_as_float(0x7fffffffu);
  } else if (to >= 0 && lane < LANES) {
    *reinterpret_cast<uint4*>(s.pool + to * (LANES * 16) + lane * 16) = piece.x[0];
  }
}
template <bool Q8>
__device__ __forceinline__ void load_new(const PageParams::Side& s, const Unit& at, int lane, Piece<Q8>& piece) {
  const uint4* src = reinterpret_cast<const uint4*>(s.rows + at.b * s.sb + at.h * s.sh + at.t * s.st + lane * kChannels<Q8>);
  piece.x[0] = src[0];
  if constexpr (Q8) piece.x[1] = src[1];
}

template <int D, int DV, bool Q8>
__global__ void __launch_bounds__(kThreads) fa_cache_write_kernel(const PageParams p) {
  grid_next();
  grid_previous();
  constexpr int N = kUnroll<true, Q8>, KL = D / kChannels<Q8>, VL = DV / kChannels<Q8>, LANES = KL > VL ? KL : VL,
                ROWS = kThreads / LANES;
  const int lane = threadIdx.x % LANES, n0 = blockIdx.x * (ROWS * N) + threadIdx.x / LANES;
  Piece<Q8> k[N] = {}, v[N] = {};
  long long to[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int n = n0 + u * ROWS;
    to[u] = -1;
    if (n >= p.units) continue;
    const Unit at = unit_of(p, n);
    if (p.lengths && at.t >= __ldg(p.lengths + at.b)) continue;  // a padding token
    if (lane < KL) load_new<Q8>(p.side[0], at, lane, k[u]);
    if (lane < VL) load_new<Q8>(p.side[1], at, lane, v[u]);
    to[u] = pool_row(p, at.b, at.h, (long long)__ldg(p.starts + at.b) + at.t);
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    write_row<KL, Q8>(p.side[0], k[u], to[u], lane);
    write_row<VL, Q8>(p.side[1], v[u], to[u], lane);
  }
}

// A lane's 8 values of a row (e4m3: the codes, and the scale in z).
template <int LANES, bool Q8>
__device__ __forceinline__ uint4 load_row(const PageParams::Side& s, long long from, int lane) {
  if constexpr (!Q8) return *reinterpret_cast<const uint4*>(s.pool + from * (LANES * 16) + lane * 16);
  const uint2 c = *reinterpret_cast<const uint2*>(s.pool + from * (LANES * 8) + lane * 8);
  return make_uint4(c.x, c.y, __float_as_uint(__ldg(s.scale + from)), 0);
}
__device__ __forceinline__ uint2 bf16_of(uint32_t codes, float f) {  // four codes
  uint32_t a, b;
  float v[4];
  asm("{\n\t.reg .b16 c, u;\n\tmov.b32 {c, u}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(codes));
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}" : "=f"(v[0]), "=f"(v[1]) : "r"(a));
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}" : "=f"(v[2]), "=f"(v[3]) : "r"(b));
  return make_uint2(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f));
}
template <int LANES, bool Q8>
__device__ __forceinline__ void store_row(const PageParams::Side& s, int n, uint4 x, int lane) {
  if (lane >= LANES) return;
  if constexpr (Q8) {
    const float f = __uint_as_float(x.z);
    const uint2 a = bf16_of(x.x, f), b = bf16_of(x.y, f);
    x = make_uint4(a.x, a.y, b.x, b.y);
  }
  *reinterpret_cast<uint4*>(s.rows + (long long)n * (LANES * 8) + lane * 8) = x;
}

template <int D, int DV, bool Q8>
__global__ void __launch_bounds__(kThreads) fa_cache_read_kernel(const PageParams p) {
  grid_next();
  grid_previous();
  constexpr int N = kUnroll<false, Q8>, KL = D / 8, VL = DV / 8, LANES = KL > VL ? KL : VL, ROWS = kThreads / LANES;
  const int lane = threadIdx.x % LANES, n0 = blockIdx.x * (ROWS * N) + threadIdx.x / LANES;
  uint4 k[N], v[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int n = n0 + u * ROWS;
    k[u] = v[u] = make_uint4(0, 0, 0, 0);
    if (n >= p.units) continue;
    const Unit at = unit_of(p, n);
    if (at.t >= __ldg(p.lengths + at.b)) continue;
    const long long from = pool_row(p, at.b, at.h, at.t);
    if (from < 0) continue;
    if (lane < KL) k[u] = load_row<KL, Q8>(p.side[0], from, lane);
    if (lane < VL) v[u] = load_row<VL, Q8>(p.side[1], from, lane);
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int n = n0 + u * ROWS;
    if (n >= p.units) continue;
    store_row<KL, Q8>(p.side[0], n, k[u], lane);
    store_row<VL, Q8>(p.side[1], n, v[u], lane);
  }
}

// ---------------------------------------------------------------- join
// Adds up the parts of each output row, in their order: those of its own keys and those
// of its group's prefix.  WARPS warps take a row (1, or 4 where there are few rows: a
// long sequence alone has tens of parts).
// All that does not depend on one another is loaded together: a row's time is that of its
// chain of loads (heads and groups, then parts, four at a time).
template <int DV, int WARPS>
__global__ void __launch_bounds__(128) fa_cache_join_kernel(const fa::CacheJoin j) {
  constexpr int CH = DV / 32;
  __shared__ float s_o[4][DV], s_ml[4][2];
  grid_next();
  grid_previous();
  const CacheParams& p = j.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int out = blockIdx.x * (4 / WARPS) + warp / WARPS;
  if (out >= p.B * p.Hq * p.T) return;  // (with WARPS 4 a block has one row)
  const int sub = warp % WARPS;
  const int bh = p.by_T(out), t = out - bh * p.T, b = j.by_Hq(bh), hq = bh - b * p.Hq, h = j.by_G(hq), g = hq - h * p.G;
  const fa::CacheHead own_head = p.parts.head[j.own + b];
  const int own_per = p.parts.head[j.own_entries].work;
  // The group of this sequence, if it has a prefix.
  fa::CacheHead pre_head = {0, 0, 0};
  int pre_per = 1, bundle = 1, first = 0, pre_rows = 0;
  if (p.S) {
    pre_per = j.pre.head[j.pre_entries].work;
    bundle = j.pre.head[j.pre_entries].item;
    for (int s0 = 0; s0 < p.S; s0 += 32) {
      const int s = s0 + lane;
      int a = 0, z = 0;
      fa::CacheHead head = {0, 0, 0};
      if (s < p.S) {
        fa::cache_group(p, s, &a, &z);
        head = j.pre.head[s];
      }
      const unsigned found = __ballot_sync(~0u, a <= b && b < z && head.chunks > 0);
      if (found) {
        const int src = __ffs(found) - 1;
        first = __shfl_sync(~0u, a, src);
        pre_rows = (__shfl_sync(~0u, z, src) - first) * p.G * p.T;
        pre_head = {__shfl_sync(~0u, head.work, src), __shfl_sync(~0u, head.item, src), __shfl_sync(~0u, head.chunks, src)};
        break;
      }
    }
  }
  const CacheSlots own = fa::cache_slots(own_head, p.G * p.T, kCacheRows, p.own_item, 1, h, g * p.T + t, own_per);
  if (!p.S && own.n == 1) return;  // a whole item, stored by its CTA
  const int pre_row = (b - first) * p.G * p.T + g * p.T + t;
  const CacheSlots pre =
      fa::cache_slots(pre_head, pre_rows, j.pre_rows, j.pre_rows == kCacheRows ? p.own_item : fa::kPrefixItem, bundle, h, pre_row, pre_per);
  // A prefix's item of at most 128 rows leaves two parts, 128 rows apart.
  const int halves = j.pre_rows == fa::kPrefixRows && pre_rows - (pre_row - pre.row) <= fa::kPrefixRows / 2 ? 1 : 0;
  const int pre_n = pre.n << halves, n = own.n + pre_n;
  float top = -INFINITY, sum = 0.f, acc[CH] = {};
  for (int i0 = sub * 4; i0 < n; i0 += WARPS * 4) {
    float2 ml[4];
    float v[4][CH];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k;
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int x = 0; x < CH; ++x) v[k][x] = 0.f;
      if (i >= n) continue;
      const bool is_pre = i < pre_n;
      const long long row = is_pre ? (pre.slot + (i >> halves) * pre.step) * j.pre_rows + pre.row + (i & halves) * 128
                                   : (own.slot + i - pre_n) * kCacheRows + own.row;
      ml[k] = reinterpret_cast<const float2*>(is_pre ? j.pre.ml : p.parts.ml)[row];
      const float* o = (is_pre ? j.pre.part : p.parts.part) + row * DV + lane * CH;
      if constexpr (CH == 4) {
        const float4 x = *reinterpret_cast<const float4*>(o);
        v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(o);
        v[k][0] = x.x, v[k][1] = x.y;
      }
    }
    const float now = fmaxf(top, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));
    const float a = top == now ? 1.f : ex2(top - now);
    top = now;
    sum *= a;
#pragma unroll
    for (int x = 0; x < CH; ++x) acc[x] *= a;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = ml[k].x == -INFINITY ? 1.f : ex2(ml[k].x - top);  // (without a finite reference, O is 0 or NaN)
      sum += ml[k].y * f;
#pragma unroll
      for (int x = 0; x < CH; ++x) acc[x] += v[k][x] * f;
    }
  }
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int k = 0; k < CH; ++k) s_o[sub][lane * CH + k] = acc[k];
    if (lane == 0) s_ml[sub][0] = top, s_ml[sub][1] = sum;
    __syncthreads();
    if (sub) return;
    top = fmaxf(fmaxf(s_ml[0][0], s_ml[1][0]), fmaxf(s_ml[2][0], s_ml[3][0]));
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) acc[k] = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = s_ml[w][0] == -INFINITY ? 1.f : ex2(s_ml[w][0] - top);
      sum += s_ml[w][1] * f;
#pragma unroll
      for (int k = 0; k < CH; ++k) acc[k] += s_o[w][lane * CH + k] * f;
    }
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t w[CH / 2];
#pragma unroll
  for (int k = 0; k < CH; k += 2) w[k / 2] = pack_bf16x2(acc[k] * f, acc[k + 1] * f);
  uint16_t* dst = p.O + (long long)out * DV + lane * CH;
  if constexpr (CH == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = w[0];
  if (lane == 0) p.L[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------- host
bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Sizes that all three calls share.
fa_status check_cache_dims(const fa_cache_dims* dims) {
  if (!dims) return FA_ERR_INVALID_ARG;
  const fa_cache_dims& z = *dims;
  if (z.B < 0 || z.Hkv < 0 || z.T < 0 || z.d < 1 || z.dv < 1 || z.pages < 0 || z.page < 1 || z.table_pages < 0)
    return FA_ERR_INVALID_ARG;
  if (z.quantised != 0 && z.quantised != 1) return FA_ERR_INVALID_ARG;
  if ((z.d != 64 && z.d != 128) || (z.dv != 64 && z.dv != 128)) return FA_ERR_UNSUPPORTED;
  if (z.page < 16 || z.page > 256 || (z.page & (z.page - 1))) return FA_ERR_UNSUPPORTED;
  if ((long long)z.table_pages * z.page > (1 << 30) || z.T > (1 << 30)) return FA_ERR_UNSUPPORTED;
  if ((long long)z.B * z.Hkv > INT_MAX || (long long)z.B * z.Hkv * z.T > (1 << 30) || (long long)z.pages * z.Hkv > INT_MAX)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

fa_status check_pools(const fa_cache_dims& z, const fa_kv_cache* c) {
  if (!c) return FA_ERR_INVALID_ARG;
  if (z.pages == 0 || z.Hkv == 0) return FA_OK;
  if (!c->K || !c->V || !aligned(c->K, 16) || !aligned(c->V, 16)) return FA_ERR_INVALID_ARG;
  if (z.quantised && (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

int log2_of(int page) {
  int n = 0;
  while ((1 << n) < page) ++n;
  return n;
}

PageParams page_params(const fa_cache_dims& z, const fa_kv_cache& c, const int* tables, const int* lengths) {
  PageParams p = {};
  p.tables = tables;
  p.lengths = lengths;
  p.B = z.B;
  p.H = z.Hkv;
  p.T = z.T;
  p.cols = z.table_pages;
  p.pages = z.pages;
  p.page_log2 = log2_of(z.page);
  p.side[0].pool = static_cast<uint8_t*>(c.K);
  p.side[1].pool = static_cast<uint8_t*>(c.V);
  p.side[0].scale = c.k_scale;
  p.side[1].scale = c.v_scale;
  p.units = z.B * z.Hkv * z.T;
  p.by_inner = fa::Divide::of(z.T);
  p.by_outer = fa::Divide::of(z.Hkv);
  p.status = fa::device_status_word();
  return p;
}

template <typename Kernel>
fa_status launch_pages(Kernel kernel, const fa_cache_dims& z, const PageParams& p, int channels, int unroll, void* stream) {
  const int lanes = (z.d > z.dv ? z.d : z.dv) / channels;
  const int per = kThreads / lanes * unroll, blocks = (p.units + per - 1) / per;
  return fa::launch_next(kernel, dim3((unsigned)blocks), kThreads, 0, static_cast<cudaStream_t>(stream), p) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

// Checks what the attention's sizes have to be besides; on success its shape.
fa_status attn_shape(const fa_cache_dims& z, const fa_cache_prefix* pre, fa::CacheShape* s) {
  if (z.Hq < 0 || (z.Hq > 0 && (z.Hkv < 1 || z.Hq % z.Hkv))) return FA_ERR_INVALID_ARG;
  const int S = pre ? pre->groups : 0, p_cols = pre ? pre->table_pages : 0;
  if (S < 0 || p_cols < 0) return FA_ERR_INVALID_ARG;
  if ((long long)p_cols * z.page > (1 << 30)) return FA_ERR_UNSUPPORTED;
  // rows are counted in 32 bits, those of a whole group among them
  const long long rows = z.Hkv ? (long long)(z.Hq / z.Hkv) * z.T : 0;
  if ((long long)z.B * z.Hq > INT_MAX || rows * z.B > (1 << 30) || (long long)z.B * z.Hq * z.T > (1 << 30))
    return FA_ERR_UNSUPPORTED;
  const int sms = fa::sm_count() > 0 ? fa::sm_count() : 1;  // (without a device the launch fails)
  *s = fa::cache_shape(z.B, z.Hkv, rows, z.dv, z.quantised, (long long)z.table_pages * z.page, S, (long long)p_cols * z.page, sms);
  return !s->fits || (long long)S + z.B > (1 << 30) ? FA_ERR_UNSUPPORTED : FA_OK;
}

}  // namespace

namespace fa {

template <int DV>
static cudaError_t launch_join(const CacheJoin& j, cudaStream_t stream) {
  const long long rows = (long long)j.p.B * j.p.Hq * j.p.T;
  // Four warps a row where there are few: only a long sequence among few has many parts.
  if (rows <= 512) return launch_next(fa_cache_join_kernel<DV, 4>, dim3((unsigned)rows), 128, 0, stream, j);
  return launch_next(fa_cache_join_kernel<DV, 1>, dim3((unsigned)((rows + 3) / 4)), 128, 0, stream, j);
}

cudaError_t launch_cache_join(const CacheJoin& j, int dv, cudaStream_t stream) {
  return dv == 64 ? launch_join<64>(j, stream) : launch_join<128>(j, stream);
}

}  // namespace fa

extern "C" {

fa_status fa_cache_write(const fa_cache_dims* dims, const fa_kv_cache* cache, const void* K, const void* V,
                         const long long* k_stride, const long long* v_stride, const int* tables, const int* starts,
                         const int* counts, void* stream) {
  fa_status e = check_cache_dims(dims);
  if (e != FA_OK || (e = check_pools(*dims, cache)) != FA_OK) return e;
  if (!k_stride || !v_stride) return FA_ERR_INVALID_ARG;
  const fa_cache_dims& z = *dims;
  if ((long long)z.B * z.Hkv * z.T == 0) return FA_OK;
  for (int k = 0; k < 3; ++k)
    if (k_stride[k] % 8 || v_stride[k] % 8) return FA_ERR_INVALID_ARG;
  if (!K || !V || !aligned(K, 16) || !aligned(V, 16) || !starts || !aligned(starts, 4) || !aligned(counts, 4) ||
      (z.table_pages && !tables) || !aligned(tables, 4))
    return FA_ERR_INVALID_ARG;
  PageParams p = page_params(z, *cache, tables, counts);
  if (!p.status) return FA_ERR_CUDA;
  p.starts = starts;
  // The rows as they lie: of a packed projection a token's heads are neighbours.
  if (z.Hkv > 1 && k_stride[1] < k_stride[2]) {
    p.heads_first = 1;
    p.by_inner = fa::Divide::of(z.Hkv);
    p.by_outer = fa::Divide::of(z.T);
  }
  const void* rows[2] = {K, V};
  const long long* strides[2] = {k_stride, v_stride};
  for (int k = 0; k < 2; ++k) {
    p.side[k].rows = static_cast<uint16_t*>(const_cast<void*>(rows[k]));
    p.side[k].sb = strides[k][0];
    p.side[k].sh = strides[k][1];
    p.side[k].st = strides[k][2];
  }
  auto pick = [&](auto q8) {
    constexpr bool Q = decltype(q8)::value;
    return z.d == 64 ? (z.dv == 64 ? fa_cache_write_kernel<64, 64, Q> : fa_cache_write_kernel<64, 128, Q>)
                     : (z.dv == 64 ? fa_cache_write_kernel<128, 64, Q> : fa_cache_write_kernel<128, 128, Q>);
  };
  return z.quantised ? launch_pages(pick(std::true_type{}), z, p, kChannels<true>, kUnroll<true, true>, stream)
                     : launch_pages(pick(std::false_type{}), z, p, kChannels<false>, kUnroll<true, false>, stream);
}

fa_status fa_cache_read(const fa_cache_dims* dims, const fa_kv_cache* cache, const int* tables, const int* lengths,
                        void* K, void* V, void* stream) {
  fa_status e = check_cache_dims(dims);
  if (e != FA_OK || (e = check_pools(*dims, cache)) != FA_OK) return e;
  const fa_cache_dims& z = *dims;
  if ((long long)z.B * z.Hkv * z.T == 0) return FA_OK;
  if (!K || !V || !aligned(K, 16) || !aligned(V, 16) || !lengths || !aligned(lengths, 4) || (z.table_pages && !tables) ||
      !aligned(tables, 4))
    return FA_ERR_INVALID_ARG;
  PageParams p = page_params(z, *cache, tables, lengths);
  if (!p.status) return FA_ERR_CUDA;
  p.side[0].rows = static_cast<uint16_t*>(K);
  p.side[1].rows = static_cast<uint16_t*>(V);
  auto pick = [&](auto q8) {
    constexpr bool Q = decltype(q8)::value;
    return z.d == 64 ? (z.dv == 64 ? fa_cache_read_kernel<64, 64, Q> : fa_cache_read_kernel<64, 128, Q>)
                     : (z.dv == 64 ? fa_cache_read_kernel<128, 64, Q> : fa_cache_read_kernel<128, 128, Q>);
  };
  return launch_pages(z.quantised ? pick(std::true_type{}) : pick(std::false_type{}), z, p, 8, kUnroll<false, false>, stream);
}

size_t fa_cache_attention_workspace_bytes(const fa_cache_dims* dims, const fa_cache_prefix* prefix) {
  fa::CacheShape s;
  if (check_cache_dims(dims) != FA_OK || attn_shape(*dims, prefix, &s) != FA_OK) return 0;
  return (long long)dims->B * dims->Hq * dims->T == 0 ? 0 : s.total;
}

fa_status fa_cache_attention(const fa_cache_dims* dims, const fa_kv_cache* cache, const fa_cache_scores* scores,
                             const fa_cache_prefix* prefix, const void* Q, const int* tables, const int* lengths, void* O,
                             float* L, void* workspace, size_t workspace_bytes, void* stream) {
  fa_status e = check_cache_dims(dims);
  if (e != FA_OK || (e = check_pools(*dims, cache)) != FA_OK) return e;
  const fa_cache_dims& z = *dims;
  fa::CacheShape s;
  if ((e = attn_shape(z, prefix, &s)) != FA_OK) return e;
  const int S = prefix ? prefix->groups : 0, p_cols = prefix ? prefix->table_pages : 0;
  fa_cache_scores sc = {};
  if (scores) sc = *scores;
  if (!(sc.scale == sc.scale) || std::isinf(sc.scale) || sc.window < 0) return FA_ERR_INVALID_ARG;
  if (sc.softcap != 0.f && !(sc.softcap >= 0x1p-10f && sc.softcap <= 0x1p10f)) return FA_ERR_INVALID_ARG;
  if (!aligned(sc.slopes, 4)) return FA_ERR_INVALID_ARG;
  // distances stay exact in fp32, as for fa_scores
  if (sc.slopes && (long long)(z.table_pages + p_cols) * z.page > (1 << 24)) return FA_ERR_UNSUPPORTED;
  if ((long long)z.B * z.Hq * z.T == 0) return FA_OK;
  if (!Q || !O || !L || !lengths || !aligned(Q, 16) || !aligned(O, 16) || !aligned(L, 4) || !aligned(lengths, 4) ||
      (z.table_pages && !tables) || !aligned(tables, 4))
    return FA_ERR_INVALID_ARG;
  if (S && (!prefix->lengths || (p_cols && !prefix->tables) || !aligned(prefix->tables, 4) || !aligned(prefix->lengths, 4) ||
              !aligned(prefix->starts, 4) || (S > 1 && !prefix->starts)))
    return FA_ERR_INVALID_ARG;
  if (s.total && (!workspace || !aligned(workspace, 256) || workspace_bytes < s.total)) return FA_ERR_INVALID_ARG;
  fa::CacheParams p = {};
  p.status = fa::device_status_word();
  if (!p.status) return FA_ERR_CUDA;
  p.Q = static_cast<const uint16_t*>(Q);
  // (a pool without pages may have no address; nothing is read of it, and Q's stands in)
  const bool none = z.pages == 0;
  p.K = static_cast<const uint8_t*>(none ? Q : cache->K);
  p.V = static_cast<const uint8_t*>(none ? Q : cache->V);
  p.k_scale = none ? static_cast<const float*>(Q) : cache->k_scale;
  p.v_scale = none ? static_cast<const float*>(Q) : cache->v_scale;
  p.tables = tables;
  p.lengths = lengths;
  if (S) {
    p.p_tables = prefix->tables;
    p.p_lengths = prefix->lengths;
    p.p_starts = prefix->starts;
  }
  p.slopes = sc.slopes;
  p.O = static_cast<uint16_t*>(O);
  p.L = L;
  p.B = z.B;
  p.Hq = z.Hq;
  p.Hkv = z.Hkv;
  p.G = z.Hq / z.Hkv;
  p.T = z.T;
  p.by_T = fa::Divide::of(p.T);
  p.by_GT = fa::Divide::of(p.G * p.T);
  p.pages = z.pages;
  p.page_log2 = log2_of(z.page);
  p.cols = z.table_pages;
  p.S = S;
  p.p_cols = p_cols;
  // a window of all keys and more hides nothing
  p.window = sc.window >= ((long long)z.table_pages + p_cols) * z.page ? 0 : sc.window;
  const float scale = sc.scale > 0.f ? sc.scale : 1.0f / std::sqrt((float)z.d);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.capped = sc.softcap > 0.f;
  p.cap = fa::cap_params(sc.softcap, scale);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto parts_of = [ws](const fa::CacheList& l) {
    return fa::CacheParts{reinterpret_cast<fa::CacheHead*>(ws + l.head), reinterpret_cast<float*>(ws + l.ml),
                          reinterpret_cast<float*>(ws + l.part)};
  };
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t err = cudaSuccess;
  p.joined = S > 0;
  p.own_item = fa::cache_item(fa::cache_few((long long)p.G * p.T, S > 0 && !s.apart));
  p.whole = s.whole;
  fa::CacheJoin j = {};
  j.pre = parts_of(s.pre);
  fa::CacheParams pre = {};
  if (s.apart) {
    p.sms = fa::sm_count();
    p.groups = S;
    p.per_sm = fa::cache_ctas(z.quantised, fa::cache_few(p.G * p.T, false));
    p.chunk_cost = fa::cache_chunk_cost(z.d, z.dv, z.quantised);
    pre = p;
    pre.parts = j.pre;
    pre.entries = S;
    pre.min_chunks = fa::kPrefixMinChunks;
    pre.max_items = (int)s.pre.items;
    pre.look = reinterpret_cast<int*>(ws + s.look);
    err = z.quantised ? fa::launch_cache_prefix_e4m3(pre, z.d, z.dv, s.pre.grid, st)
                      : fa::launch_cache_prefix_bf16(pre, z.d, z.dv, s.pre.grid, st);
    if (err != cudaSuccess) return FA_ERR_CUDA;
    p.S = 0;
  }
  p.parts = parts_of(s.list);
  p.entries = p.S + z.B;
  p.min_chunks = fa::kCacheMinChunks;
  p.max_items = (int)s.list.items;
  err = z.quantised ? fa::launch_cache_attn_e4m3(p, z.d, z.dv, s.list.grid, st)
                    : fa::launch_cache_attn_bf16(p, z.d, z.dv, s.list.grid, st);
  if (err == cudaSuccess && s.apart && !z.quantised && p.window)
    err = fa::launch_cache_prefix_careful(pre, z.d, z.dv, s.pre.grid, st);
  if (s.whole) return err == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  j.p = p;
  j.p.S = S;
  j.own = p.S;
  j.by_Hq = fa::Divide::of(z.Hq);
  j.by_G = fa::Divide::of(p.G);
  j.own_entries = p.entries;
  j.pre_rows = s.apart ? fa::kPrefixRows : kCacheRows;
  j.pre_entries = s.apart ? S : p.entries;
  if (err == cudaSuccess) err = fa::launch_cache_join(j, z.dv, st);
  return err == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
