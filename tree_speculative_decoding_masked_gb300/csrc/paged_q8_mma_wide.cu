// Paged attention of few rows over pages in 8 bits, heads of more than 128: paged_mma.cuh's kernel.
#include "paged_mma.cuh"

namespace tv {

cudaError_t launch_pm_q8_wide(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const PmPlan& p,
                              cudaStream_t stream) {
  return launch_pm_d<256, true>(mk, mv, a, p, stream);
}

}  // namespace tv
