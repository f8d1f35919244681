// Forward pass: the plain instances of the kernel in fa_fwd_kernel.cuh and the
// launcher that picks an instance (the score-modified ones are compiled in
// fa_scored_64.cu and fa_scored_128.cu).
#include "fa_fwd_kernel.cuh"

namespace {

template <int HD, int HDV>
cudaError_t launch_fwd_dims(const fa::Problem& pr, const CUtensorMap& mq, const CUtensorMap& mk,
                            const CUtensorMap& mv, void* O, float* L, cudaStream_t stream) {
  if (!pr.causal) return launch_fwd_t<HD, HDV, false, false, fa::kPlain>(pr, {}, mq, mk, mv, O, L, stream);
  if (pr.window) return launch_fwd_t<HD, HDV, true, true, fa::kPlain>(pr, {}, mq, mk, mv, O, L, stream);
  return launch_fwd_t<HD, HDV, true, false, fa::kPlain>(pr, {}, mq, mk, mv, O, L, stream);
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
                           void* O, float* L, cudaStream_t stream, int* launches) {
  const long long rows = (long long)pr.B * pr.Hq * pr.Tq;
  if (rows == 0) return cudaSuccess;
  if (pr.Tk == 0) {
    const size_t words = (size_t)rows * pr.dv / 2;
    fa_fwd_empty_keys<<<1216, 256, 0, stream>>>(static_cast<uint32_t*>(O), words, L, (size_t)rows);
    ++*launches;
    return cudaGetLastError();
  }
  CUtensorMap mq, mk, mv;
  if (!encode_rows_bf16(&mq, Q, pr.d, pr.Tq, (long long)pr.B * pr.Hq) ||
      !encode_rows_bf16(&mk, K, pr.d, pr.Tk, (long long)pr.B * pr.Hkv) ||
      !encode_rows_bf16(&mv, V, pr.dv, pr.Tk, (long long)pr.B * pr.Hkv))
    return cudaErrorInvalidValue;
  cudaError_t e;
  if (mods.any())
    e = pr.d == 64 ? launch_fwd_scored_64(pr, mods, mq, mk, mv, O, L, stream)
                   : launch_fwd_scored_128(pr, mods, mq, mk, mv, O, L, stream);
  else if (pr.d == 64)
    e = pr.dv == 64 ? launch_fwd_dims<64, 64>(pr, mq, mk, mv, O, L, stream)
                    : launch_fwd_dims<64, 128>(pr, mq, mk, mv, O, L, stream);
  else
    e = pr.dv == 64 ? launch_fwd_dims<128, 64>(pr, mq, mk, mv, O, L, stream)
                    : launch_fwd_dims<128, 128>(pr, mq, mk, mv, O, L, stream);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace fa
