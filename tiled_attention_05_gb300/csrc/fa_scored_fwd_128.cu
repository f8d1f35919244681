// Score-modified forward instances (fa_fwd_kernel.cuh) with Q and K heads of 128.
#include "fa_fwd_kernel.cuh"

namespace {

template <int HDV>
cudaError_t launch_dims(const fa::Problem& p, const fa::ScoreMods& m, const CUtensorMap& mq, const CUtensorMap& mk,
                        const CUtensorMap& mv, void* O, float* L, cudaStream_t stream) {
  switch (m.fwd_bits()) {
    case 0:
      return launch_fwd_t<128, HDV, false, false, 0>(p, m, mq, mk, mv, O, L, stream);
    case fa::kCap:
      return launch_fwd_t<128, HDV, false, false, fa::kCap>(p, m, mq, mk, mv, O, L, stream);
    case fa::kCap | fa::kBounded:
      return launch_fwd_t<128, HDV, false, false, fa::kCap | fa::kBounded>(p, m, mq, mk, mv, O, L, stream);
    case fa::kCap | fa::kSlopes | fa::kBounded:
      return launch_fwd_t<128, HDV, false, false, fa::kCap | fa::kSlopes | fa::kBounded>(p, m, mq, mk, mv, O, L, stream);
    case fa::kSlopes:
      return launch_fwd_t<128, HDV, false, false, fa::kSlopes>(p, m, mq, mk, mv, O, L, stream);
  }
  return launch_fwd_t<128, HDV, false, false, fa::kCap | fa::kSlopes>(p, m, mq, mk, mv, O, L, stream);
}

}  // namespace

cudaError_t fa::launch_fwd_scored_128(const Problem& p, const ScoreMods& m, const CUtensorMap& mq, const CUtensorMap& mk,
                                     const CUtensorMap& mv, void* O, float* L, cudaStream_t stream) {
  return p.dv == 64 ? launch_dims<64>(p, m, mq, mk, mv, O, L, stream)
                    : launch_dims<128>(p, m, mq, mk, mv, O, L, stream);
}
