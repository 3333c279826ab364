// cache_attn_256.cu -- cache_attn_kernel for head dimension 256.
#include "cache_attn.cuh"

namespace lbx {
namespace cache {
template <>
cudaError_t launch_attn<256>(bool f16, const AttnMaps &maps, const AttnArgs &A, int grid,
                             cudaStream_t stream) {
  if (A.til.ctas == 2)
    return f16 ? launch_attn_of<256, true, true>(maps, A, grid, stream)
               : launch_attn_of<256, false, true>(maps, A, grid, stream);
  return f16 ? launch_attn_of<256, true, false>(maps, A, grid, stream)
             : launch_attn_of<256, false, false>(maps, A, grid, stream);
}
}  // namespace cache
}  // namespace lbx
