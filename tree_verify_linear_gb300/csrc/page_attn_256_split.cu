// page_attn_256_split.cu -- page_attn_kernel for head dimension 256, weights in two parts.
#include "page_attn.cuh"

namespace lbx {
namespace paged {
template <>
cudaError_t launch_page_attn<256, false, true>(bool f16, const PageMaps &maps, const PageArgs &A, int grid,
                                         cudaStream_t stream) {
  return f16 ? launch_page_attn_of<256, true, false, true>(maps, A, grid, stream)
             : launch_page_attn_of<256, false, false, true>(maps, A, grid, stream);
}
}  // namespace paged
}  // namespace lbx
