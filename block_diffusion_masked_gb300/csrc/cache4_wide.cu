// Attention over the paged 4-bit cache for many rows to a key, headdim 64 (more than 32) and
// 128: the kernel of cache_wide.cuh for 4 bits.
#include "cache_wide.cuh"

namespace dfa {

cudaError_t launch_cache_wide(const Cache4FwdParams& p, int headdim, cudaStream_t stream) {
  if (headdim == 64) return launch_wide<4, 64, 6>(p, stream);
  if (headdim == 128) return launch_wide<4, 128, 3>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace dfa
