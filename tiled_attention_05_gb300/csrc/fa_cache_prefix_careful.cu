// The prefix kernel of bf16 caches for shares in whose results a NaN or an infinity was found.
#include "fa_cache_prefix.cuh"

namespace fa {

cudaError_t launch_cache_prefix_careful(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream) {
  return launch_prefix<false, true>(p, d, dv, grid, stream);
}

}  // namespace fa
