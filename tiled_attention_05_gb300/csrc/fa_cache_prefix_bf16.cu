// Shared prefixes of bf16 caches (see fa_cache_prefix.cuh).
#include "fa_cache_prefix.cuh"

namespace fa {

cudaError_t launch_cache_prefix_bf16(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream) {
  return p.window ? launch_cache_prefix_window(p, d, dv, grid, stream) : launch_prefix<false, false, false>(p, d, dv, grid, stream);
}

}  // namespace fa
