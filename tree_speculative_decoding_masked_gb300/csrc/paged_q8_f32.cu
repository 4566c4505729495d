// Paged attention over 8-bit pages on CUDA cores: paged_f32.cuh's kernel with codes for K and V.
#include "paged_f32.cuh"

namespace tv {

cudaError_t launch_paged_q8_f32(PagedAttn a, char* ws, tv_dtype dtype, cudaStream_t stream) {
  return dtype == TV_BF16 ? launch_pf_d<true, uint16_t>(a, ws, stream) : launch_pf_d<true, float>(a, ws, stream);
}

}  // namespace tv
