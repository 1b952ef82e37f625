// The tile kernel over a cache in E4M3 (paged_tiles.cuh).
#include "paged_tiles.cuh"

namespace fa {

cudaError_t launch_tiles_fp8(const PagedTiles& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                             const CUtensorMap& tm_v, int d, int ctas, cudaStream_t stream) {
  return launch_any<true>(p, tm_q, tm_k, tm_v, d, ctas, stream);
}

}  // namespace fa
