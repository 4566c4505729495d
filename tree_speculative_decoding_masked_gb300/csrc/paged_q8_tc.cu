// Paged attention of many rows over pages in 8 bits: paged_tc.cuh's kernel.
#include "paged_tc.cuh"

namespace tv {

cudaError_t launch_paged_q8_tc(PagedAttn a, char* ws, cudaStream_t stream) { return launch_pt_all<true>(a, ws, stream); }

}  // namespace tv
