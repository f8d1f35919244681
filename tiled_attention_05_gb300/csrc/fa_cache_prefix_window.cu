// Shared prefixes of bf16 caches with a window (see fa_cache_prefix.cuh): the kernel, and the one
// for shares in whose results a NaN or an infinity was found.
#include "fa_cache_prefix.cuh"

namespace fa {

cudaError_t launch_cache_prefix_window(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream) {
  return launch_prefix<false, true, false>(p, d, dv, grid, stream);
}
cudaError_t launch_cache_prefix_careful(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream) {
  return launch_prefix<false, true, true>(p, d, dv, grid, stream);
}

}  // namespace fa
