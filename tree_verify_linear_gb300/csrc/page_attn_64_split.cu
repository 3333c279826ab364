// page_attn_64_split.cu -- page_attn_kernel for head dimension 64, weights in two parts.
#include "page_attn.cuh"

namespace lbx {
namespace paged {
template <>
cudaError_t launch_page_attn<64, false, true>(bool f16, const PageMaps &maps, const PageArgs &A, int grid,
                                         cudaStream_t stream) {
  return f16 ? launch_page_attn_of<64, true, false, true>(maps, A, grid, stream)
             : launch_page_attn_of<64, false, false, true>(maps, A, grid, stream);
}
}  // namespace paged
}  // namespace lbx
