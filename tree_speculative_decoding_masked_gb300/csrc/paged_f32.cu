// Paged attention of many fp32 rows over fp32 pages: paged_f32.cuh's kernel.
#include "paged_f32.cuh"

namespace tv {

PagedWs paged_f32_ws(int B, int Hq, int Hkv, int D, int N) {
  const size_t n = pf_plan(B, Hq, Hkv, D, N, paged_device_sms()).bytes;
  return {n, n};
}

cudaError_t launch_paged_f32(PagedAttn a, char* ws, cudaStream_t stream) {
  return launch_pf_d<false>(a, ws, stream);
}

}  // namespace tv
