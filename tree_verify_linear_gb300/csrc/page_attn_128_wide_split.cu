// page_attn_128_wide_split.cu -- page_attn_kernel for head dimension 128, pairs of CTAs, weights in two parts.
#include "page_attn.cuh"

namespace lbx {
namespace paged {
template <>
cudaError_t launch_page_attn<128, true, true>(bool f16, const PageMaps &maps, const PageArgs &A, int grid,
                                         cudaStream_t stream) {
  return f16 ? launch_page_attn_of<128, true, true, true>(maps, A, grid, stream)
             : launch_page_attn_of<128, false, true, true>(maps, A, grid, stream);
}
}  // namespace paged
}  // namespace lbx
