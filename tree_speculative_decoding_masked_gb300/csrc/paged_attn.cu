// Paged attention's entry: the kernel for a call.
//   fp32, more than 16 query rows a KV head  paged_f32_kernel (row tiles on CUDA cores)
//   fp32, at most 4                          paged_rows_kernel (keys over the warps)
//   other fp32                               paged_simt_kernel (a row or two a warp)
//   bf16, more than 16 query rows a KV head,
//     D <= 128, G <= 16                      paged_tc_kernel (row tiles on tcgen05)
//   other bf16                               paged_mma_kernel (a stream of keys past few rows)
// 64 sequences of 8192 to 16384 tokens, G = 4: at 16 rows (4 nodes) the stream takes 486 us and
// row tiles 539; at 32 (8 nodes) the stream's warp-level products set the pace, 768 us against
// 540.  Over 500 to 1000 tokens 75 against 69 us at 16 rows and 115 against 69 at 32; one sequence
// of 2048 12.0 against 11.5 and 15.2 against 11.5: the rule gives short ranges' 5 % for long ones' 10.
#include <atomic>

#include "paged.cuh"

namespace tv {

int paged_device_sms() {
  static std::atomic<int> known[64];  // 0 = not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  int n = known[dev].load(std::memory_order_relaxed);
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return min(n, kPagedMaxSms);
}

int paged_grid_sms() {
  const int n = paged_device_sms(), share = sm_share_attention();
  return share > 0 && share < n ? share : n;
}

static bool f32_tiles(int Hq, int Hkv, int N) { return (long long)(Hq / Hkv) * N > kPagedFewRows; }

PagedWs paged_attn_ws(int B, int Hq, int Hkv, int D, int N, tv_dtype dtype, int sms) {
  if (dtype == TV_F32) return f32_tiles(Hq, Hkv, N) ? paged_f32_ws(B, Hq, Hkv, D, N) : paged_simt_ws(D);
  return paged_tc_takes(Hq, Hkv, D, N) ? paged_tc_ws(B, Hq, Hkv, D, N) : paged_mma_ws(B, Hq, Hkv, D, N, sms);
}

cudaError_t launch_paged_attn(PagedAttn a, tv_dtype dtype, char* ws, cudaStream_t stream) {
  if (dtype == TV_F32)
    return f32_tiles(a.Hq, a.Hkv, a.N) ? launch_paged_f32(a, ws, stream) : launch_paged_simt(a, ws, stream);
  return paged_tc_takes(a.Hq, a.Hkv, a.D, a.N) ? launch_paged_tc(a, ws, stream) : launch_paged_mma(a, ws, stream);
}

}  // namespace tv
