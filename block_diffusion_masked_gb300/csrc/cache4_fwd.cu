// Attention over the paged 4-bit cache, up to 32 rows to a key, and headdim 256: the
// kernel of cache_rows.cuh for 4 bits.
#include "cache_rows.cuh"

namespace dfa {

cudaError_t launch_cache4_rows(const Cache4FwdParams& p, int headdim, int tile_rows,
                               cudaStream_t stream) {
  return headdim == 64    ? launch_cache_rows<4, 64>(p, tile_rows, stream)
         : headdim == 128 ? launch_cache_rows<4, 128>(p, tile_rows, stream)
                          : launch_cache_rows<4, 256>(p, tile_rows, stream);
}

}  // namespace dfa
