// Score-modified backward instances (fa_bwd_kernel.cuh) with Q and K heads of 64.
#include "fa_bwd_kernel.cuh"

namespace {

template <int HDV>
cudaError_t launch_dims(const fa::Problem& p, const fa::ScoreMods& m, const CUtensorMap* maps, const ScoredBwdParams& bp,
                        cudaStream_t stream) {
  switch (m.bits()) {
    case 0:
      return launch_main_t<64, HDV, false, false, 0>(p, maps, bp, stream);
    case fa::kCap:
      return launch_main_t<64, HDV, false, false, fa::kCap>(p, maps, bp, stream);
    case fa::kSlopes:
      return launch_main_t<64, HDV, false, false, fa::kSlopes>(p, maps, bp, stream);
  }
  return launch_main_t<64, HDV, false, false, fa::kCap | fa::kSlopes>(p, maps, bp, stream);
}

}  // namespace

cudaError_t fa::launch_bwd_scored_64(const Problem& p, const ScoreMods& m, const CUtensorMap* maps, const ScoredBwdParams& bp,
                                     cudaStream_t stream) {
  return p.dv == 64 ? launch_dims<64>(p, m, maps, bp, stream) : launch_dims<128>(p, m, maps, bp, stream);
}
