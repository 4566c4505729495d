// Paged attention of many rows over pages in 8 bits: paged_tc.cuh's kernel.
#include "paged_tc.cuh"

namespace tv {

cudaError_t launch_paged_q8_tc(PagedAttn a, char* ws, cudaStream_t stream) {
  return a.block_shift >= 4 ? launch_pt_all<kPtQ8>(a, ws, stream) : launch_pt_all<kPtQ8Fine>(a, ws, stream);
}

}  // namespace tv
