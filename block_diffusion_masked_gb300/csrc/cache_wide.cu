// Attention over the paged 8-bit cache for more than 32 rows to a key, headdim 64 and
// 128: the kernel of cache_wide.cuh for 8 bits.
#include "cache_wide.cuh"

namespace dfa {

cudaError_t launch_cache_wide(const CacheFwdParams& p, int headdim, cudaStream_t stream) {
  if (headdim == 64) return launch_wide<8, 64, 6>(p, stream);
  if (headdim == 128) return launch_wide<8, 128, 2>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace dfa
