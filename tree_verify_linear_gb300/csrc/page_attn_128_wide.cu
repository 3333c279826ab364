// page_attn_128_wide.cu -- page_attn_kernel for head dimension 128, pairs of CTAs.
#include "page_attn.cuh"

namespace lbx {
namespace paged {
template <>
cudaError_t launch_page_attn<128, true, false>(bool f16, const PageMaps &maps, const PageArgs &A, int grid,
                                         cudaStream_t stream) {
  return f16 ? launch_page_attn_of<128, true, true, false>(maps, A, grid, stream)
             : launch_page_attn_of<128, false, true, false>(maps, A, grid, stream);
}
}  // namespace paged
}  // namespace lbx
