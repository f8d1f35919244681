// fa_cache_attention over e4m3 caches (see fa_cache_attn.cuh).
#include "fa_cache_attn.cuh"

namespace fa {

cudaError_t launch_cache_attn_e4m3(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream) {
  return launch_cache<true>(p, d, dv, grid, stream);
}

}  // namespace fa
