// fa_cache_attention over bf16 caches (see fa_cache_attn.cuh).
#include "fa_cache_attn.cuh"

namespace fa {

cudaError_t launch_cache_attn_bf16(const CacheParams& p, int d, int dv, int grid, cudaStream_t stream) {
  return launch_cache<false>(p, d, dv, grid, stream);
}

}  // namespace fa
