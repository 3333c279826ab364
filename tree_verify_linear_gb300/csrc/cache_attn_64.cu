// cache_attn_64.cu -- cache_attn_kernel for head dimension 64.
#include "cache_attn.cuh"

namespace lbx {
namespace cache {
template <>
cudaError_t launch_attn<64>(bool f16, const AttnMaps &maps, const AttnArgs &A, int grid,
                             cudaStream_t stream) {
  return f16 ? launch_attn_of<64, true, false>(maps, A, grid, stream)
             : launch_attn_of<64, false, false>(maps, A, grid, stream);
}
}  // namespace cache
}  // namespace lbx
