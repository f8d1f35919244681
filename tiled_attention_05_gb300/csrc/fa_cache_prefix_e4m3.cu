// Shared prefixes of e4m3 caches (see fa_cache_prefix.cuh).
#include "fa_cache_prefix.cuh"

namespace fa {

cudaError_t launch_cache_prefix_e4m3(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream) {
  return p.window ? launch_prefix<true, true, false>(p, d, dv, grid, stream) : launch_prefix<true, false, false>(p, d, dv, grid, stream);
}

}  // namespace fa
