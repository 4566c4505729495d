// Paged attention of many rows over bf16 pages: paged_tc.cuh's kernel.  And what it shares with that over 8-bit
// pages: tensor maps and the schedule.
#include "paged_tc.cuh"

namespace tv {

typedef CUresult (*PtEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static bool pt_encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                      const cuuint32_t* box, CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  static std::atomic<PtEncodeFn> known{nullptr};
  PtEncodeFn fn = known.load(std::memory_order_relaxed);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    fn = reinterpret_cast<PtEncodeFn>(p);
    known.store(fn, std::memory_order_relaxed);
  }
  const cuuint32_t step[5] = {1, 1, 1, 1, 1};
  return fn(m, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// rows [planes][rows][D] as boxes of 64 columns x box_rows
static bool pt_tmap(CUtensorMap* m, const void* base, int D, int rows, long long planes, int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)rows * D * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  return pt_encode(m, base, 3, dims, strides, box);
}

bool paged_kv_tmap(CUtensorMap* m, const void* base, const PagedAttn& a) {
  const int ps = 1 << a.page_shift, box = min(ps, 64);
  const long long planes = (long long)a.num_pages * a.Hkv;
  if (a.D == 128 || a.D == 256) {
    // {64 columns, 8 rows, column blocks, row groups, planes}
    const cuuint64_t blocks = (cuuint64_t)a.D / 64;
    const cuuint64_t dims[5] = {64, 8, blocks, (cuuint64_t)ps / 8, (cuuint64_t)planes};
    const cuuint64_t strides[4] = {(cuuint64_t)a.D * 2, 128, (cuuint64_t)a.D * 16, (cuuint64_t)ps * a.D * 2};
    const cuuint32_t boxes[5] = {64, 8, (cuuint32_t)blocks, (cuuint32_t)box / 8, 1};
    return pt_encode(m, base, 5, dims, strides, boxes);
  }
  // one column block, or a narrower last one: then a box is one 8-row group of a block
  return pt_tmap(m, base, a.D, ps, planes, a.D <= 64 ? box : 8);
}

bool paged_q_tmap(CUtensorMap* m, const PagedAttn& a, int rows) {
  return pt_tmap(m, a.q, a.D, a.N, (long long)a.B * a.Hq, rows);
}

bool paged_q8_tmap(CUtensorMap* m, const void* base, const PagedAttn& a, PagedQ8Box kind, int rows) {
  const int ps = 1 << a.page_shift, box = min(ps, rows);
  const cuuint64_t planes = (cuuint64_t)a.num_pages * a.Hkv, D = (cuuint64_t)a.D;
  const CUtensorMapSwizzle swizzle = kind == kQ8Rows128   ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : kind == kQ8Swizzled ? CU_TENSOR_MAP_SWIZZLE_64B
                                                           : CU_TENSOR_MAP_SWIZZLE_NONE;
  const cuuint32_t cols = kind == kQ8Rows128 ? 128 : 64;
  const bool one = a.D <= (int)cols;  // column block, or less of one: zeros behind
  if (!one && (a.D == 128 || a.D == 256)) {
    // {columns, 8 rows, column blocks, row groups, planes}
    const cuuint64_t dims[5] = {cols, 8, D / cols, (cuuint64_t)ps / 8, planes};
    const cuuint64_t strides[4] = {D, cols, D * 8, (cuuint64_t)ps * D};
    const cuuint32_t boxes[5] = {cols, 8, (cuuint32_t)(a.D / cols), (cuuint32_t)box / 8, 1};
    return pt_encode(m, base, 5, dims, strides, boxes, CU_TENSOR_MAP_DATA_TYPE_UINT8, swizzle);
  }
  // else a box is one 8-row group of a block
  const cuuint64_t dims[3] = {D, (cuuint64_t)ps, planes};
  const cuuint64_t strides[2] = {D, (cuuint64_t)ps * D};
  const cuuint32_t boxes[3] = {cols, (cuuint32_t)(one ? box : 8), 1};
  return pt_encode(m, base, 3, dims, strides, boxes, CU_TENSOR_MAP_DATA_TYPE_UINT8, swizzle);
}

// Clusters of s CTAs that can be resident at once on the current device (known per device and s).
static int pt_clusters(int D, int s) {
  static std::atomic<int> known[64][kPtMaxSplits + 1];  // count + 1; 0 = not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return paged_device_sms() / s;
  int n = known[dev][s].load(std::memory_order_relaxed) - 1;
  if (n < 0) {
    // every instance takes one CTA per SM, so one stands for all
    const void* fn = reinterpret_cast<const void*>(paged_tc_kernel<128, kNoCap, false, kPtBf16>);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s * 64, 1, 1);
    cfg.blockDim = dim3(PtCfg<128, kPtBf16>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = PtCfg<128, kPtBf16>::kSmemAlloc;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)s;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, PtCfg<128, kPtBf16>::kSmemAlloc) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess)
      n = paged_device_sms() / s;
    known[dev][s].store(n + 1, std::memory_order_relaxed);
  }
  return n;
}

PtPlan paged_tc_plan(int B, int Hq, int Hkv, int D, int N, int share) {
  PtPlan p{};
  const int G = Hq / Hkv;
  p.NT = (kPtRows / G) / 8 * 8;
  const int sms = paged_device_sms(), row_tiles = (N + p.NT - 1) / p.NT;
  // the most parts that leave all units resident on `on` SMs at once: of single tiles, of pairs
  auto parts = [&](int tiles, int on) -> int {
    const long long units = (long long)B * Hkv * ((row_tiles + tiles - 1) / tiles);
    if (units * 2 > on || B > 65535 || Hkv > 65535) return 0;
    for (int s = kPtMaxSplits; s >= 2; --s)
      if (units * s <= on && units <= pt_clusters(D, s)) return s;
    return 0;
  };
  const int one = parts(1, sms), two = parts(2, sms);
  // Single tiles merge half the rows, 2 us less, but read K and V once for each: a 64-key step of 64 CTAs
  // takes 0.75 us, of 128 1.0, a pair's 0.8.  32 heads over 8, single / pair: 64 nodes (8 parts either
  // way) over 512 tokens 10.4 / 12.4 us, 2048 12.8 / 14.7, 8192 24.8 / 24.1, 32768 73.5 / 64.0; 128 nodes
  // (4 parts or 8) 12.0 / 13.9, 16.0 / 17.0, 34.0 / 29.7, 107 / 83; 96 nodes (6 or 8) 11.6 / 13.6,
  // 14.7 / 16.5, 28.9 / 29.3, 87.6 / 81.6.  Lengths are not known here: the rule goes by short ranges
  // where the parts are nearly as many, and gives long ones up to 15 %
  p.tiles = one >= 2 && one * 4 >= two * 3 ? 1 : 2;
  p.splits = p.tiles == 1 ? one : two;
  p.MP = (row_tiles + p.tiles - 1) / p.tiles;
  // one part per CTA of the clusters, two per CTA of the persistent grid
  p.slots = p.splits ? (size_t)p.splits * p.MP * B * Hkv : (size_t)2 * kPagedMaxSms;
  if (p.splits && share < sms) {
    // on a share: fewer parts of the same units, else of pairs, else the persistent grid.  The workspace stays
    // the whole device's, which holds them: pairs have parts <= share < 2 units of single tiles
    p.splits = parts(p.tiles, share);
    if (!p.splits) {
      p.tiles = 2;
      p.splits = parts(2, share);
      p.MP = (row_tiles + 1) / 2;
    }
  }
  p.grid = (int)min((size_t)share, p.slots / 2);
  p.bytes = kPagedCntBytes + p.slots * 2 * kPtRows * (8 + (D <= 64 ? 64 : 128) * 4);
  return p;
}

bool paged_tc_takes(int Hq, int Hkv, int D, int N) {
  const int G = Hq / Hkv;
  return D <= 128 && G <= 16 && (long long)G * N > kPagedFewRows;
}

PagedWs paged_tc_ws(int B, int Hq, int Hkv, int D, int N) {
  const size_t n = paged_tc_plan(B, Hq, Hkv, D, N, paged_device_sms()).bytes;
  return {n, n};
}

cudaError_t launch_paged_tc(PagedAttn a, char* ws, cudaStream_t stream) { return launch_pt_all<kPtBf16>(a, ws, stream); }

}  // namespace tv
