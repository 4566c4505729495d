// Paged attention of fp32 rows over 8-bit pages, on CUDA cores: paged_rows.cuh's kernel for at most four query
// rows of a KV head, paged_f32.cuh's for more.
#include "paged_f32.cuh"
#include "paged_rows.cuh"

namespace tv {

static bool q8_few(int Hq, int Hkv, int N) { return (long long)(Hq / Hkv) * N <= 4; }

PagedWs paged_q8_f32_ws(int B, int Hq, int Hkv, int D, int N) {
  return q8_few(Hq, Hkv, N) ? paged_simt_ws(D) : paged_f32_ws(B, Hq, Hkv, D, N);
}

cudaError_t launch_paged_q8_f32(PagedAttn a, char* ws, cudaStream_t stream) {
  return q8_few(a.Hq, a.Hkv, a.N) ? launch_paged_rows<true>(a, ws, stream) : launch_pf_d<true>(a, ws, stream);
}

}  // namespace tv
