// Paged attention of few rows over bf16 pages: paged_mma.cuh's kernel.
#include "paged_mma.cuh"

namespace tv {

PagedWs paged_mma_ws(int B, int Hq, int Hkv, int D, int N, int sms) {
  const PmPlan p = pm_plan(B, Hq, Hkv, D, N, sms);
  return {p.bytes, p.splits ? 0 : p.bytes};
}

cudaError_t launch_paged_mma(PagedAttn a, char* ws, cudaStream_t stream) { return launch_pm_all<false>(a, ws, stream); }

}  // namespace tv
