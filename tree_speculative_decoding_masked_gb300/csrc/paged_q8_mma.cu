// Paged attention of few rows over pages in 8 bits: paged_mma.cuh's kernel (heads of more than 128:
// paged_q8_mma_wide.cu).
#include "paged_mma.cuh"

namespace tv {

cudaError_t launch_paged_q8_mma(PagedAttn a, char* ws, cudaStream_t stream) { return launch_pm_all<true>(a, ws, stream); }

}  // namespace tv
