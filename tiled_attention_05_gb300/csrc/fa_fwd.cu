// Forward pass: the plain instances of the kernel in fa_fwd_kernel.cuh and the
// launcher that picks an instance (the score-modified ones are compiled in
// fa_scored_fwd_*.cu).
#include "fa_fwd_kernel.cuh"

namespace {

template <int HD, int HDV>
cudaError_t launch_fwd_dims(const fa::Problem& pr, const fa::FwdShape& shape, const CUtensorMap& mq,
                            const CUtensorMap& mk, const CUtensorMap& mv, void* O, float* L, cudaStream_t stream) {
  constexpr int S = fa::kPlain;
  if (!pr.causal) return launch_fwd_t<HD, HDV, false, false, S>(pr, {}, shape, mq, mk, mv, O, L, nullptr, stream);
  if (pr.window) return launch_fwd_t<HD, HDV, true, true, S>(pr, {}, shape, mq, mk, mv, O, L, nullptr, stream);
  return launch_fwd_t<HD, HDV, true, false, S>(pr, {}, shape, mq, mk, mv, O, L, nullptr, stream);
}

// Joins the parts of a split forward: with reference m_s and sum l_s of part s and
// M = max m_s, O = sum 2^(m_s - M) O_s over the same sum of what each O is divided by,
// and L = ln2 (M + log2 sum 2^(m_s - M) l_s).  A part without a key tile has l = -1 and
// no O.  One whose weights are all 0 counts with factor 0 (its O is 0, or NaN from a NaN
// in V), and a NaN sum makes O and L NaN, both as in an unsplit row.  One warp a row,
// HDV / 32 columns a lane.  Bound by HBM / L2 (the parts, fp32) and by its launch.
template <int HDV>
__global__ void __launch_bounds__(256) fa_fwd_join(const float* __restrict__ part, uint16_t* __restrict__ O,
                                                   float* __restrict__ L, long long rows, int rows_per_head,
                                                   int pairs, int n_bh, int split, long long n_parts) {
  grid_next();
  grid_previous();
  constexpr int W = HDV / 32;
  const long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const long long bh = row / rows_per_head;
  const int i = (int)(row - bh * rows_per_head);
  const int pair = pairs - 1 - i / (2 * BM);  // (items take the last pair first, heads fastest)
  const long long first = ((long long)pair * n_bh + bh) * split;  // the item's first part
  const int at = i % (2 * BM);
  const float4* ml = reinterpret_cast<const float4*>(part + n_parts * 2 * BM * HDV);
  float top = -__int_as_float(0x7f800000);
  for (int s = lane; s < split; s += 32) {
    const float4 v = ml[(first + s) * 2 * BM + at];
    if (v.y > 0.f || v.y != v.y) top = fmaxf(top, v.x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  float sum = 0.f, sum_o = 0.f, acc[W];
#pragma unroll
  for (int e = 0; e < W; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int s = 0; s < split; ++s) {
    const float4 v = ml[(first + s) * 2 * BM + at];
    if (v.y < 0.f) continue;
    const float w = v.y == 0.f ? 0.f : exp2f(v.x - top);
    const float* o = part + ((first + s) * 2 * BM + at) * HDV + lane * W;
    sum += w * v.y;
    sum_o += w * v.z;
#pragma unroll
    for (int e = 0; e < W; ++e) acc[e] += w * o[e];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum_o;
  uint32_t* out = reinterpret_cast<uint32_t*>(O + row * HDV + lane * W);
#pragma unroll
  for (int e = 0; e < W; e += 2) out[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) L[row] = sum == 0.f ? -__int_as_float(0x7f800000) : (top + log2f(sum)) * 0.69314718055994531f;
}

__global__ void fa_fwd_empty_keys(uint32_t* O_words, size_t n_words, float* L, size_t n_rows) {
  const float NEG_INF = -__int_as_float(0x7f800000);
  for (size_t t = blockIdx.x * (size_t)blockDim.x + threadIdx.x; t < n_words || t < n_rows;
       t += (size_t)gridDim.x * blockDim.x) {
    if (t < n_words) O_words[t] = 0u;
    if (t < n_rows) L[t] = NEG_INF;
  }
}

}  // namespace

namespace fa {

cudaError_t launch_forward(const Problem& pr, const ScoreMods& mods, const void* Q, const void* K, const void* V,
                           void* O, float* L, void* workspace, size_t workspace_bytes, cudaStream_t stream,
                           int* launches) {
  const long long rows = (long long)pr.B * pr.Hq * pr.Tq;
  if (rows == 0) return cudaSuccess;
  if (pr.Tk == 0) {
    const size_t words = (size_t)rows * pr.dv / 2;
    fa_fwd_empty_keys<<<1216, 256, 0, stream>>>(static_cast<uint32_t*>(O), words, L, (size_t)rows);
    ++*launches;
    return cudaGetLastError();
  }
  FwdShape shape = fwd_shape(pr, mods, sm_count());
  float* part = static_cast<float*>(workspace);
  if (shape.split > 1 && (!part || workspace_bytes < fwd_workspace_bytes(pr, shape))) shape.split = 1;
  CUtensorMap mq, mk, mv;
  if (!encode_rows_bf16(&mq, Q, pr.d, shape.rows, (long long)pr.B * shape.heads) ||
      !encode_rows_bf16(&mk, K, pr.d, pr.Tk, (long long)pr.B * pr.Hkv) ||
      !encode_rows_bf16(&mv, V, pr.dv, pr.Tk, (long long)pr.B * pr.Hkv))
    return cudaErrorInvalidValue;
  cudaError_t e;
  if (mods.any()) {
    const FwdLauncher go = shape.few() ? (pr.d == 64 ? fwd_scored_few_64(pr, mods) : fwd_scored_few_128(pr, mods))
                                       : (pr.d == 64 ? fwd_scored_64(pr, mods) : fwd_scored_128(pr, mods));
    e = go(pr, mods, shape, mq, mk, mv, O, L, part, stream);
  } else if (pr.d == 64)
    e = pr.dv == 64 ? launch_fwd_dims<64, 64>(pr, shape, mq, mk, mv, O, L, stream)
                    : launch_fwd_dims<64, 128>(pr, shape, mq, mk, mv, O, L, stream);
  else
    e = pr.dv == 64 ? launch_fwd_dims<128, 64>(pr, shape, mq, mk, mv, O, L, stream)
                    : launch_fwd_dims<128, 128>(pr, shape, mq, mk, mv, O, L, stream);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (shape.split > 1) {
    auto join = pr.dv == 64 ? fa_fwd_join<64> : fa_fwd_join<128>;
    const int pairs = (shape.rows + 2 * BM - 1) / (2 * BM);
    e = launch_next(join, (unsigned)((rows + 7) / 8), 256, 0, stream, part, static_cast<uint16_t*>(O), L, rows, shape.rows,
                    pairs, pr.B * shape.heads, shape.split, shape.items * shape.split);
    if (e == cudaSuccess) ++*launches;
  }
  return e;
}

}  // namespace fa
