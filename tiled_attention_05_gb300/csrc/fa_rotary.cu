// Rotary positions of Q and K, with one to four position axes.
//
// Frequency f (of rot / 2) belongs to the axis a(f) whose section holds it; it
// turns channel pair f of token (b, t) by the angle
//     theta = positions[a(f)][b][t] * inv_freq[f]:
//     (x, y) -> (x cos theta - y sin theta, y cos theta + x sin theta),
// the same for every head.  The gradient of a rotation is the rotation by
// -theta.  Pair f is channels (f, f + rot/2), or (2f, 2f + 1) when interleaved;
// channels from rot on are copied.
//
// Angles.  Only the fraction of a turn matters, so it is taken exactly: the
// turns per step, inv_freq / 2 pi, are a 64-bit fixed-point fraction F (from
// inv_freq's 24-bit significand times 2^64 / 2 pi), and positions * F modulo
// 2^64 drops whole turns for free.  The error is |position| * 2^-64 turns at
// most for |inv_freq| <= 1, so far positions lose nothing.  The upper 32 bits,
// as a signed fraction of half a turn, go to sincospif.  (The same in double
// precision costs ~4 FP64 operations per angle at ~2 per clock and SM.)
//
// Mapping.  Bound by HBM: every element is read once and written once.  A
// thread owns 16 channels (8 pairs) of one token, turns its angles into 16
// registers once and walks the heads, two 16-byte loads and stores each, so
// the angles cost nothing per head and no shared memory is needed.  Few
// tokens are spread over the SMs by giving each block a share of the heads.
// Small blocks, six an SM, four heads in flight a thread, and shares of whole
// rounds of four were the best of a sweep (T 8192, B 2, 32 + 8 heads of 128, 335 MB:
// 53.5 us, 92% of the measured copy rate, against 60.5 with blocks of 256 and any
// share; B 3, T 4099, 32 heads of 64, half turned, 101 MB: 16.7 against 23.8).
// Inputs may be strided (views of a packed [B, T, heads * d] projection); the
// output strides are the caller's too.
#include <climits>
#include <cmath>
#include <cstdint>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

using namespace fa_ptx;

namespace {

constexpr int kThreads = 128;
constexpr int kUnit = 16;  // channels per thread
constexpr int kUnroll = 4;  // heads in flight per thread

struct Strides {
  long long b, h, t;
};

struct RotaryParams {
  const uint16_t *q, *k;
  uint16_t *qo, *ko;
  Strides sq, sk, sqo, sko;
  const void* pos;
  long long pos_axis, pos_batch;
  int pos64;
  const float* inv_freq;
  long long tokens;  // B * T
  int T, Hq, heads, rot;
  int heads_per_block;
  int sec_end[3];  // first frequency of axis 1, 2, 3 (rot / 2 where there is none)
  int inverse;
};

// Turns per position step of one frequency: frac(f / 2 pi) * 2^64.
__device__ __forceinline__ uint64_t turns_per_step(float f) {
  const uint32_t bits = __float_as_uint(f);
  const int ex = (int)((bits >> 23) & 255u);
  const uint64_t m = ex ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int e = (ex ? ex : 1) - 150;  // |f| = m * 2^e
  constexpr uint64_t kInv2Pi = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi)
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  uint64_t r;
  if (e >= 0)
    r = e < 64 ? lo << e : 0ull;
  else if (e > -64)
    r = (lo >> -e) | (hi << (64 + e));
  else
    r = e > -128 ? hi >> (-64 - e) : 0ull;
  return (bits >> 31) ? 0ull - r : r;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// UNITS: threads per token (d / 16).
template <int UNITS, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 6) fa_rotary_kernel(const RotaryParams p) {
  grid_next();
  grid_previous();
  const long long n = (long long)blockIdx.x * (kThreads / UNITS) + threadIdx.x / UNITS;
  if (n >= p.tokens) return;
  const int unit = threadIdx.x % UNITS;
  const long long b = n / p.T, t = n - b * p.T;
  const int half = p.rot >> 1;
  const bool turn = unit * kUnit < p.rot;
  // the two 8-channel chunks of this thread
  const int c0 = (turn && !INTERLEAVED) ? unit * 8 : unit * kUnit;
  const int c1 = (turn && !INTERLEAVED) ? c0 + half : c0 + 8;
  const long long q_at = b * p.sq.b + t * p.sq.t, k_at = b * p.sk.b + t * p.sk.t;
  const long long qo_at = b * p.sqo.b + t * p.sqo.t, ko_at = b * p.sko.b + t * p.sko.t;
  const int h0 = blockIdx.y * p.heads_per_block, h1 = min(p.heads, h0 + p.heads_per_block);

  auto load = [&](int h, uint4& x, uint4& y) {
    const uint16_t* src = h < p.Hq ? p.q + q_at + h * p.sq.h : p.k + k_at + (h - p.Hq) * p.sk.h;
    x = *reinterpret_cast<const uint4*>(src + c0);
    y = *reinterpret_cast<const uint4*>(src + c1);
  };
  uint4 x[kUnroll], y[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (h0 + u < h1) load(h0 + u, x[u], y[u]);

  float cs[8], sn[8];
  if (turn) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int f = unit * 8 + e;
      const int axis = (f >= p.sec_end[0]) + (f >= p.sec_end[1]) + (f >= p.sec_end[2]);
      const long long at = axis * p.pos_axis + b * p.pos_batch + t;
      const long long pos = p.pos64 ? static_cast<const long long*>(p.pos)[at] : static_cast<const int*>(p.pos)[at];
      const uint64_t turns = (uint64_t)pos * turns_per_step(p.inv_freq[f]);
      sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &sn[e], &cs[e]);
      if (p.inverse) sn[e] = -sn[e];
    }
  }

  for (int h = h0; h < h1; h += kUnroll) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u >= h1) break;
      uint32_t a[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, c[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
      if (turn) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if (INTERLEAVED) {  // each word is a pair: words of chunk 0 are pairs 0..3, of chunk 1 pairs 4..7
            const float a0 = bf_lo(a[w]), a1 = bf_hi(a[w]), b0 = bf_lo(c[w]), b1 = bf_hi(c[w]);
            a[w] = pack_bf16x2(a0 * cs[w] - a1 * sn[w], a1 * cs[w] + a0 * sn[w]);
            c[w] = pack_bf16x2(b0 * cs[w + 4] - b1 * sn[w + 4], b1 * cs[w + 4] + b0 * sn[w + 4]);
          } else {  // word w holds channels 2w, 2w + 1 of both halves
            const float a0 = bf_lo(a[w]), a1 = bf_hi(a[w]), b0 = bf_lo(c[w]), b1 = bf_hi(c[w]);
            a[w] = pack_bf16x2(a0 * cs[2 * w] - b0 * sn[2 * w], a1 * cs[2 * w + 1] - b1 * sn[2 * w + 1]);
            c[w] = pack_bf16x2(b0 * cs[2 * w] + a0 * sn[2 * w], b1 * cs[2 * w + 1] + a1 * sn[2 * w + 1]);
          }
        }
      }
      const int hh = h + u;
      uint16_t* dst = hh < p.Hq ? p.qo + qo_at + hh * p.sqo.h : p.ko + ko_at + (hh - p.Hq) * p.sko.h;
      *reinterpret_cast<uint4*>(dst + c0) = make_uint4(a[0], a[1], a[2], a[3]);
      *reinterpret_cast<uint4*>(dst + c1) = make_uint4(c[0], c[1], c[2], c[3]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + kUnroll + u < h1) load(h + kUnroll + u, x[u], y[u]);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A tensor of heads x T rows per batch: pointer and strides fit 16-byte accesses.
bool ok_tensor(const void* p, const long long* s, long long elems) {
  if (elems == 0) return true;
  return p && aligned16(p) && s[0] % 8 == 0 && s[1] % 8 == 0 && s[2] % 8 == 0;
}

}  // namespace

extern "C" {

fa_status fa_rotary(const fa_rotary_dims* dims, const void* Q, const void* K, const void* positions,
                    const float* inv_freq, void* Qo, void* Ko, int inverse, void* stream) {
  if (!dims) return FA_ERR_INVALID_ARG;
  const fa_rotary_dims& z = *dims;
  if (z.B < 0 || z.Hq < 0 || z.Hk < 0 || z.T < 0 || z.d < 1 || z.rot < 0 || z.rot > z.d) return FA_ERR_INVALID_ARG;
  if (z.axes < 1 || z.axes > 4 || (z.interleaved != 0 && z.interleaved != 1) || (inverse != 0 && inverse != 1) ||
      (z.pos_bytes != 4 && z.pos_bytes != 8))
    return FA_ERR_INVALID_ARG;
  long long sum = 0;
  for (int a = 0; a < z.axes; ++a) {
    if (z.section[a] < 0) return FA_ERR_INVALID_ARG;
    sum += z.section[a];
  }
  if (2 * sum != z.rot) return FA_ERR_INVALID_ARG;
  if ((z.d != 64 && z.d != 128) || z.rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  const long long tokens = (long long)z.B * z.T, heads = (long long)z.Hq + z.Hk;
  const int units = z.d / kUnit, per_block = kThreads / units;
  if (heads > 65535 || (tokens + per_block - 1) / per_block > INT_MAX) return FA_ERR_UNSUPPORTED;
  if (tokens == 0 || heads == 0) return FA_OK;
  if (!ok_tensor(Q, z.q_stride, z.Hq) || !ok_tensor(Qo, z.qo_stride, z.Hq) || !ok_tensor(K, z.k_stride, z.Hk) ||
      !ok_tensor(Ko, z.ko_stride, z.Hk))
    return FA_ERR_INVALID_ARG;
  if (z.rot > 0 && (!positions || !inv_freq || (reinterpret_cast<uintptr_t>(positions) & (z.pos_bytes - 1)) ||
                    (reinterpret_cast<uintptr_t>(inv_freq) & 3u)))
    return FA_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    return FA_ERR_CUDA;
  RotaryParams p;
  p.q = static_cast<const uint16_t*>(Q);
  p.k = static_cast<const uint16_t*>(K);
  p.qo = static_cast<uint16_t*>(Qo);
  p.ko = static_cast<uint16_t*>(Ko);
  p.sq = {z.q_stride[0], z.q_stride[1], z.q_stride[2]};
  p.sk = {z.k_stride[0], z.k_stride[1], z.k_stride[2]};
  p.sqo = {z.qo_stride[0], z.qo_stride[1], z.qo_stride[2]};
  p.sko = {z.ko_stride[0], z.ko_stride[1], z.ko_stride[2]};
  p.pos = positions;
  p.pos_axis = z.pos_axis_stride;
  p.pos_batch = z.pos_batch_stride;
  p.pos64 = z.pos_bytes == 8;
  p.inv_freq = inv_freq;
  p.tokens = tokens;
  p.T = z.T;
  p.Hq = z.Hq;
  p.heads = (int)heads;
  p.rot = z.rot;
  p.inverse = inverse;
  int end = 0;
  for (int a = 0; a < 3; ++a) {
    end += a < z.axes ? z.section[a] : 0;
    p.sec_end[a] = a + 1 < z.axes ? end : INT_MAX;
  }
  // Enough blocks to fill the GPU several times over, each with whole rounds of
  // kUnroll heads.
  const long long xb = (tokens + per_block - 1) / per_block, want = 16LL * sms;
  long long split = xb >= want ? 1 : (want + xb - 1) / xb;
  if (split > heads) split = heads;
  p.heads_per_block = (int)((heads + split - 1) / split);
  p.heads_per_block = (p.heads_per_block + kUnroll - 1) / kUnroll * kUnroll;
  const dim3 grid((unsigned)xb, (unsigned)((heads + p.heads_per_block - 1) / p.heads_per_block));
  auto kernel = z.d == 64 ? (z.interleaved ? fa_rotary_kernel<4, true> : fa_rotary_kernel<4, false>)
                          : (z.interleaved ? fa_rotary_kernel<8, true> : fa_rotary_kernel<8, false>);
  return fa::launch_next(kernel, grid, kThreads, 0, static_cast<cudaStream_t>(stream), p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
