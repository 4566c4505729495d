// Attention of few rows over a paged KV cache (single tokens, short chunks, small trees), bf16.
//
// With few query rows a KV head every key is read for a handful of products: the
// work is a stream of K and V pages from HBM and the kernel's job is to keep enough of
// them in flight.  Four warps fetch 64-key tiles by TMA (a box per page piece, dealt to them
// in turn: one warp's issue of the 8 boxes of 16-row pages took 0.65 us a tile, as long as
// an SM's share of HBM takes to bring them) into a ring and run ahead across sequences and
// heads; groups of four warps take the tiles in turn, a warp 16 keys of a tile, by warp-level
// MMAs on shared memory:
//   S^T = K Q^T  (16 keys x 8 rows a product),  O^T += V^T P^T  (16 columns x 8 rows).
// With the rows on the products' short side their number follows R / 8: at 4 rows a
// 128-column tile costs a warp 16 MMAs, where rows on the long side would take 32 (and a
// tcgen05 product a 128-row tile); S^T becomes P^T's operand by movmatrix, in registers.  Each
// warp keeps its own running reference and sums (32 bits) and its own O; P is rounded to
// bf16 for the second product.  The warps' O's are added in warp order when the unit ends,
// so results do not depend on timing.
//
// Two schedules.  Units (sequence, KV head, row tile) up to half the SMs run as one cluster
// each, whose CTAs take equal parts of the unit's keys and merge through distributed shared
// memory (the copies of short and long units share the memory system, so ragged lengths
// cost little).  More units are divided equally, tile by tile, over a persistent grid
// (paged.cuh), and the parts of cut units merged through the workspace.
#include "paged.cuh"

namespace tv {

constexpr int kPmKeys = 64;
constexpr int kPmProducers = 4;
constexpr int kPmMaxSplits = 8;  // portable cluster size
constexpr int kPmMerge = 8;      // parts whose loads are in flight together
constexpr int kPmMinTiles = 2;   // tiles of a CTA's range: fewer only add parts to merge
// A unit's set-up and end count as 8 tiles, and cuts less than 8 from a unit's edge move to it
// (paged.cuh).  0 and 0 / 8 and 8: one token each of 64 sequences of 150 to 300 tokens 36.4 / 26.8 us,
// of 500 to 1000 50.8 / 46.4, of 8192 to 16384 465 / 461.
constexpr int kPmTol = 8, kPmFix = 8;

template <int kD, int kRT>
struct PmCfg {
  static constexpr int kDB = kD / 64;
  static constexpr int kNT = kRT / 8;                   // row tiles of the products
  // consumers: two groups of four; one where O takes 128 registers a thread
  static constexpr int kWarps = kD == 256 || kD / 16 * kNT * 4 > 64 ? 4 : 8;
  static constexpr int kConsumers = kWarps * 32;
  static constexpr int kThreads = kConsumers + 32 * kPmProducers;
  static constexpr int kGroup = kDB * 1024;             // 8 rows of a K or V tile: [column block][8][128 bytes]
  static constexpr int kTile = kPmKeys / 8 * kGroup;
  static constexpr int kStages = kD == 64 ? 8 : kD == 128 ? (kRT <= 16 ? 6 : 5) : 3;  // of K and V
  static constexpr int kQStride = kD * 2 + 16;          // bytes: ldmatrix rows on different banks
  static constexpr int kBatch = kD == 64 || kNT > 2 ? 4 : 8;  // K or V fragments loaded at once
  static constexpr bool kQRegs = kNT * kD <= 256;       // queries stay in registers
  // the unit's queries, masks and tree; its O at the end
  static constexpr int kOffU = kStages * 2 * kTile;
  static constexpr int kOffVis = kOffU + kRT * kQStride;
  static constexpr int kOffPar = kOffVis + kRT * (kMaxNodes / 32) * 4;
  static constexpr int kInBytes = kOffPar + kMaxNodes * 4 - kOffU;
  static constexpr int kOStride = kD + 4;               // floats: a store's four row pairs on different banks
  // warps that hand over their O at once
  static constexpr int kRegions = kD == 256 ? 1 : kD == 128 && kRT == 16 ? 2 : kWarps / 2;
  static constexpr int kOBytes = kRegions * kRT * kOStride * 4;
  static constexpr int kOffBar = kOffU + (kInBytes > kOBytes ? kInBytes : kOBytes);
  static constexpr int kSmem = kOffBar + 256 + 1024;
  // a slot's tiles alternate between no two groups: a group that skipped a slot's earlier tile
  // could take that tile's unfinished phase for its own finished one
  static_assert(kWarps == 4 || kStages % 2 == 0, "each slot belongs to one group");
  static_assert(kSmem + 8192 <= 232448,  // beside the static arrays
                "shared memory per CTA");
  static_assert(kD / 16 * kNT * 4 <= 128, "O fits in registers");
};

struct PmBars {
  uint64_t full[8];
  uint64_t empty[8];
  int abort;
};

__device__ __forceinline__ void pm_ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void pm_ldsm2(uint32_t (&r)[2], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void pm_ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t pm_transpose(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void pm_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The next unit of this CTA: of its range, or the cluster's one unit, whether it has work or not.
// The producers and the consumers walk the same sequence of them.
template <int kRT, bool kStream>
__device__ __forceinline__ bool pm_next(const PagedAttn& a, UnitWalk& w, int splits) {
  if constexpr (kStream) return unit_next(a, w, kRT, kPmKeys);
  if (w.loaded == w.b) return false;
  bool bad;
  w.loaded = w.b;
  w.P = a.prefix_len[w.b];
  w.n = paged_rows(a, w.b, w.P, &bad);
  if (w.n == 0) w.P = 0;
  if (threadIdx.x == 0 && (bad || paged_cut(a, w.b, w.P, w.n))) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
  const int T_u = unit_tiles(a, w.P, w.n, w.rt, kRT, kPmKeys), part = blockIdx.x;
  w.t0 = (int)((long long)T_u * part / splits);
  w.t1 = (int)((long long)T_u * (part + 1) / splits);
  return true;
}

template <int kD, int kRT, int kCap, bool kStream>
__global__ void __launch_bounds__(PmCfg<kD, kRT>::kThreads, 1)
    paged_mma_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, PagedAttn a,
                     int splits, int row_tiles, int wide) {
  using C = PmCfg<kD, kRT>;
  ptx::griddep_launch_dependents();
  extern __shared__ unsigned char pm_raw[];
  unsigned char* sm = pm_raw + ((1024u - (ptx::smem_addr(pm_raw) & 1023u)) & 1023u);
  PmBars* bars = reinterpret_cast<PmBars*>(sm + C::kOffBar);
  volatile int* abort_flag = &bars->abort;
  __shared__ unsigned long long s_red[kPagedRed];
  __shared__ int s_lo[kRT], s_hi[kRT], s_first_pad, s_last;
  __shared__ float s_m[C::kWarps][kRT], s_l[C::kWarps][kRT];
  __shared__ __align__(8) float2 s_ml[kRT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&bars->full[s], kPmProducers);
      ptx::mbar_init(&bars->empty[s], 4);  // one group's warps
    }
    bars->abort = 0;
    ptx::fence_mbar_init();
  }
  ptx::griddep_wait();
  __syncthreads();
  PagedSpan sp{};
  UnitWalk w{};
  w.loaded = -1;
  if constexpr (kStream) {
    sp = paged_span(a, kRT, kPmKeys, kPmMinTiles, s_red, kPmTol, kPmFix);
    __syncthreads();
    w = unit_walk(sp);
  } else {
    w.b = blockIdx.z;
    w.hk = blockIdx.y / row_tiles;
    w.rt = blockIdx.y % row_tiles;
  }
  int rows = 0, r0 = 0, n_act = 0;  // the consumers' unit
  int it = 0;  // tiles so far: ring slot it % kStages

  if (warp >= C::kWarps) {
    // ------------------------------------------------------------------ producers
    // the boxes of a tile - (row piece, column block without 5-D boxes, K or V) - dealt to the
    // producer warps in turn; lane i of a warp looks up the page of its i-th box, read a tile
    // ahead and checked when it is used
    const int per_piece = 2 * (wide ? 1 : C::kDB);
    const int box_shift = min(a.page_shift, C::kDB == 1 || wide ? 6 : 3);
    const int boxes = (kPmKeys >> box_shift) * per_piece;
    const int mine = boxes / kPmProducers + (warp - C::kWarps < boxes % kPmProducers);
    const int box = lane * kPmProducers + warp - C::kWarps;  // this lane's
    const int pi = box / per_piece, part = box % per_piece;
    const uint32_t box_bytes = (uint32_t)(256 * C::kDB / per_piece) << box_shift;
    // where it goes in a stage: K or V, 8-row group, column block
    const int off = (part & 1) * C::kTile + ((pi << box_shift) >> 3) * C::kGroup + (part >> 1) * 1024;
    int issued = 0, counted = -1, active = 0;  // a sequence's active rows, once counted
    while (pm_next<kRT, kStream>(a, w, splits)) {
      if (counted != w.b) {
        int pad = w.n;
        if (a.parent)
          for (int t = lane; t < w.n; t += 32)
            if (t > 0 && t < pad && a.parent[(size_t)w.b * a.N + t] == -1) pad = t;
        active = __reduce_min_sync(0xffffffffu, pad);
        counted = w.b;
      }
      const int unit = unit_rows(a, w.n, w.rt, kRT);
      const int lo = unit_lo(a, w.P, w.rt, kRT), tile0 = lo / kPmKeys;
      const int hi = min(w.P + active, w.P + (w.rt * kRT + unit - 1) / a.G + 1);
      const int32_t* table = a.table + (size_t)w.b * a.max_pages;
      // whether this lane's box in tile t holds a needed row, and its table entry
      auto needed = [&](int t) -> bool {
        const int j = (tile0 + t) * kPmKeys + (pi << box_shift);
        return t < w.t1 && lane < mine && j < hi && j + (1 << box_shift) > lo;
      };
      auto entry = [&](int t) -> int {
        return needed(t) ? table[((tile0 + t) * kPmKeys + (pi << box_shift)) >> a.page_shift] : 0;
      };
      int next = entry(w.t0);
      for (int t = w.t0; t < w.t1; ++t, ++it) {
        int page = needed(t) ? next : -1;
        next = entry(t + 1);
        const int slot = it % C::kStages;
        bool ok = true;
        if (it >= C::kStages) ok = ptx::mbar_wait(&bars->empty[slot], ((it / C::kStages) - 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) continue;  // aborted: no more copies; the consumers do not wait either
        issued = it + 1;
        if (needed(t) && (page < 0 || page >= a.num_pages)) {
          set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
          page = -1;
        }
        const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) ptx::mbar_arrive_expect_tx(&bars->full[slot], __popc(have) * box_bytes);
        __syncwarp();
        if (page >= 0) {
          const int row = ((tile0 + t) * kPmKeys + (pi << box_shift)) & ((1 << a.page_shift) - 1);
          unsigned char* dst = sm + slot * 2 * C::kTile + off;
          const CUtensorMap* tm = (part & 1) ? &tmV : &tmK;
          if (C::kDB > 1 && wide)
            ptx::tma_load_5d(dst, tm, &bars->full[slot], 0, 0, 0, row >> 3, page * a.Hkv + w.hk);
          else
            ptx::tma_load_3d(dst, tm, &bars->full[slot], (part >> 1) * 64, row, page * a.Hkv + w.hk);
        }
        __syncwarp();
      }
    }
    // every tile's copies have landed before the CTA ends (the consumers waited for each; after an
    // abort they did not)
    if (*abort_flag && lane == 0) {
      int quiet = 0;
      for (int s = 0; s < C::kStages && s < issued; ++s)
        ptx::mbar_wait(&bars->full[s], ((issued - 1 - s) / C::kStages) & 1, &quiet);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ consumers
    auto cons_sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(C::kConsumers) : "memory"); };
    const int wk = warp & 3, group = warp >> 2;  // key quarter of a tile, and which of two tiles in turn
    const int ct = threadIdx.x;
    unsigned char* sQ = sm + C::kOffU;
    uint32_t(*s_vis)[kMaxNodes / 32] = reinterpret_cast<uint32_t(*)[kMaxNodes / 32]>(sm + C::kOffVis);
    int* s_par = reinterpret_cast<int*>(sm + C::kOffPar);
    float* sO = reinterpret_cast<float*>(sm + C::kOffU);
    const int kg = lane >> 2, rg = (lane & 3) * 2;  // this lane's keys (columns) kg, kg + 8 and rows rg, rg + 1
    const float c = kCap == kLargeCap ? kLog2e : kCap ? a.cap * kLog2e : a.scale * kLog2e;
    const float ck = kCap == kLargeCap ? 1.f / a.cap : kCap ? 2.f * kLog2e * a.scale / a.cap : 0.f;
    bool ok = true;
    // (maximum, sum) of row rr over the warps
    auto row_max = [&](int rr) -> float {
      float M = s_m[0][rr];
#pragma unroll
      for (int k = 1; k < C::kWarps; ++k) M = fmaxf(M, s_m[k][rr]);
      return M;
    };
    auto part_ml = [&](int rr) -> float2 {
      const float M = row_max(rr);
      float L = 0.f;
#pragma unroll
      for (int k = 0; k < C::kWarps; ++k)
        if (s_m[k][rr] != -INFINITY) L = fmaf(s_l[k][rr], ptx::ex2(s_m[k][rr] - M), L);
      return make_float2(M, L);
    };
    while (pm_next<kRT, kStream>(a, w, splits)) {
      rows = unit_rows(a, w.n, w.rt, kRT);
      r0 = w.rt * kRT;
      const int lo = unit_lo(a, w.P, w.rt, kRT), tile0 = lo / kPmKeys;
      if (kStream) cons_sync();  // the previous unit's O has been read
      n_act = w.n;
      if (a.parent) {
        if (ct == 0) s_first_pad = w.n;
        cons_sync();
        int wrong = 0;
        for (int t = ct; t < w.n; t += C::kConsumers) {
          const int p = a.parent[(size_t)w.b * a.N + t];
          const bool prev_pad = t >= 2 && a.parent[(size_t)w.b * a.N + t - 1] == -1;
          const bool good = t == 0 ? p == -1 : (p == -1 || (p >= 0 && p < t && !prev_pad));
          if (!good) wrong = 1;
          s_par[t] = good ? p : -1;
          if (t > 0 && p == -1) atomicMin(&s_first_pad, t);
        }
        if (wrong) set_dev_status(a.dev_status, TV_DEV_BAD_TREE);
        cons_sync();
        n_act = s_first_pad;
      }
      const int hi = min(w.P + n_act, w.P + (r0 + rows - 1) / a.G + 1);
      for (int e = ct; e < kRT * (kD / 8); e += C::kConsumers) {
        const int rr = e / (kD / 8), ch = e % (kD / 8), i = (r0 + rr) / a.G, g = (r0 + rr) % a.G;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (rr < rows && i < n_act && ch * 8 < a.D)
          v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                              (((size_t)w.b * a.Hq + w.hk * a.G + g) * a.N + i) * a.D + ch * 8);
        *reinterpret_cast<uint4*>(sQ + rr * C::kQStride + ch * 16) = v;
      }
      if (ct < kRT) {
        // row ct sees [s_lo, s_hi) and, in a tree, its ancestors; what is no row sees everything
        const int i = (r0 + ct) / a.G;
        int wlo = 0, whi = 0x7fffffff;
        if (ct < rows && i < n_act) {
          int depth = i;
          if (a.parent) {
            whi = w.P;
            depth = -1;
            for (int k = 0; k < (w.n + 31) / 32; ++k) s_vis[ct][k] = 0u;
            for (int at = i; at >= 0; at = s_par[at]) {  // parents fall: it ends
              ++depth;
              if (a.window <= 0 || depth < a.window) s_vis[ct][at >> 5] |= 1u << (at & 31);
            }
          } else {
            whi = w.P + i + 1;
          }
          if (a.window > 0) wlo = w.P + depth - a.window + 1;
        }
        s_lo[ct] = wlo;
        s_hi[ct] = whi;
      }
      cons_sync();
      // every row sees all of [full_lo, full_hi)
      const int full_lo = __reduce_max_sync(0xffffffffu, lane < kRT ? s_lo[lane] : 0);
      const int full_hi = __reduce_min_sync(0xffffffffu, lane < kRT ? s_hi[lane] : 0x7fffffff);
      // queries as the products' B operand: rows (lane & 7), two 16-column steps a load
      const uint32_t qaddr = ptx::smem_addr(sQ + (lane & 7) * C::kQStride + (lane >> 3) * 16);
      uint32_t qf[C::kQRegs ? kD / 32 : 1][C::kNT][4];
      if constexpr (C::kQRegs) {
#pragma unroll
        for (int k2 = 0; k2 < kD / 32; ++k2)
#pragma unroll
          for (int nt = 0; nt < C::kNT; ++nt) pm_ldsm4(qf[k2][nt], qaddr + nt * 8 * C::kQStride + k2 * 64);
      }
      float o[kD / 16][C::kNT][4];
      float m[C::kNT][2], l[C::kNT][2];
#pragma unroll
      for (int nt = 0; nt < C::kNT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int k = 0; k < kD / 16; ++k)
#pragma unroll
          for (int u = 0; u < 4; ++u) o[k][nt][u] = 0.f;
      }

      for (int t = w.t0; t < w.t1; ++t, ++it) {
        if (C::kWarps == 8 && (it & 1) != group) continue;
        const int slot = it % C::kStages;
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars->full[slot], (it / C::kStages) & 1, abort_flag));
        if (!ok) continue;
        const int j0 = (tile0 + t) * kPmKeys + wk * 16;  // this warp's 16 keys
        unsigned char* sK = sm + slot * 2 * C::kTile + wk * 2 * C::kGroup;
        unsigned char* sV = sK + C::kTile;
        if (j0 >= hi || j0 + 16 <= lo) {  // none of them
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bars->empty[slot]);
          continue;
        }
        const bool edge = j0 < lo || j0 + 16 > hi;
        if (edge) {
          // V rows that were not fetched or may hold anything, NaN included: zero
          for (int e = lane; e < 16 * C::kDB * 8; e += 32) {
            const int rr = e / (C::kDB * 8), rest = e % (C::kDB * 8);
            if (j0 + rr < lo || j0 + rr >= hi)
              *reinterpret_cast<uint4*>(sV + (rr >> 3) * C::kGroup + (rest >> 3) * 1024 + (rr & 7) * 128 +
                                        (rest & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();  // before the slot is refilled
          __syncwarp();
        }
        // K as the A operand: keys (lane & 15), column chunks kk * 2 + (lane >> 4).  A batch's loads are
        // issued before its products, so that they wait for shared memory once
        const uint32_t kaddr = ptx::smem_addr(sK + ((lane >> 3) & 1) * C::kGroup + (lane & 7) * 128);
        float s[C::kNT][2][4];  // two chains each: even and odd steps
#pragma unroll
        for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
          for (int u = 0; u < 4; ++u) s[nt][0][u] = s[nt][1][u] = 0.f;
#pragma unroll
        for (int k0 = 0; k0 < kD / 16; k0 += C::kBatch) {
          uint32_t kf[C::kBatch][4];
#pragma unroll
          for (int i = 0; i < C::kBatch; ++i) {
            const int kk = k0 + i, ch = (kk & 3) * 2 + (lane >> 4);
            pm_ldsm4(kf[i], kaddr + (kk >> 2) * 1024 + ((ch ^ (lane & 7)) << 4));
          }
#pragma unroll
          for (int i = 0; i < C::kBatch; ++i) {
            const int kk = k0 + i;
#pragma unroll
            for (int nt = 0; nt < C::kNT; ++nt) {
              if constexpr (C::kQRegs) {
                pm_mma(s[nt][kk & 1], kf[i], qf[kk >> 1][nt][(kk & 1) * 2], qf[kk >> 1][nt][(kk & 1) * 2 + 1]);
              } else {
                uint32_t q2[2];
                pm_ldsm2(q2, ptx::smem_addr(sQ + (nt * 8 + (lane & 7)) * C::kQStride + kk * 32 + ((lane >> 3) & 1) * 16));
                pm_mma(s[nt][kk & 1], kf[i], q2[0], q2[1]);
              }
            }
          }
        }
        // V^T as the A operand: transposed 8 x 8 blocks of (columns, keys); the first batch is
        // fetched while the scores are turned into weights
        const uint32_t vaddr = ptx::smem_addr(sV + (lane >> 4) * C::kGroup + (lane & 7) * 128);
        uint32_t vf[C::kBatch][4];
        auto load_v = [&](int k0) {
#pragma unroll
          for (int i = 0; i < C::kBatch; ++i) {
            const int k = k0 + i, ch = (k & 3) * 2 + ((lane >> 3) & 1);
            pm_ldsm4t(vf[i], vaddr + (k >> 2) * 1024 + ((ch ^ (lane & 7)) << 4));
          }
        };
        load_v(0);
        const bool masked = j0 < full_lo || j0 + 16 > full_hi || edge;
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float z = s[nt][0][u] + s[nt][1][u];
            if constexpr (kCap == kTanhCap) z = soft_tanh(z * ck);
            if constexpr (kCap == kLargeCap) z = capped_score(z * a.scale, a.cap, ck);
            z *= c;
            if (masked) {
              const int rr = nt * 8 + rg + (u & 1), j = j0 + kg + (u >> 1) * 8;
              bool vis = j >= s_lo[rr] && j < s_hi[rr];
              if (!vis && a.parent && j >= w.P && j < hi)
                vis = (s_vis[rr][(j - w.P) >> 5] >> ((j - w.P) & 31)) & 1u;
              if (!vis) z = -INFINITY;
            }
            s[nt][0][u] = z;
            grow |= z > m[nt][u & 1] + 8.f;
          }
        // a row's running reference moves when a score exceeds it by 2^8
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(s[nt][0][e], s[nt][0][e + 2]);
#pragma unroll
              for (int x = 4; x < 32; x *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
              if (mx > m[nt][e]) {
                const float f = ptx::ex2(m[nt][e] - mx);  // 0 from -inf
                m[nt][e] = mx;
                l[nt][e] *= f;
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                  o[k][nt][e] *= f;
                  o[k][nt][e + 2] *= f;
                }
              }
            }
        }
        uint32_t pf[C::kNT][2];
#pragma unroll
        for (int nt = 0; nt < C::kNT; ++nt) {
          const float b0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], b1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
          const float e0 = ptx::ex2(s[nt][0][0] - b0), e1 = ptx::ex2(s[nt][0][1] - b1);
          const float e2 = ptx::ex2(s[nt][0][2] - b0), e3 = ptx::ex2(s[nt][0][3] - b1);
          l[nt][0] += e0 + e2;
          l[nt][1] += e1 + e3;
          pf[nt][0] = pm_transpose(ptx::cvt_bf16x2(e0, e1));
          pf[nt][1] = pm_transpose(ptx::cvt_bf16x2(e2, e3));
        }
#pragma unroll
        for (int k0 = 0; k0 < kD / 16; k0 += C::kBatch) {
          if (k0) load_v(k0);
#pragma unroll
          for (int i = 0; i < C::kBatch; ++i)
#pragma unroll
            for (int nt = 0; nt < C::kNT; ++nt) pm_mma(o[k0 + i][nt], vf[i], pf[nt][0], pf[nt][1]);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->empty[slot]);
      }

      // ---- the warps' results, added in order
#pragma unroll
      for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 4; x < 32; x *= 2) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
          if (kg == 0) {
            s_m[warp][nt * 8 + rg + e] = m[nt][e];
            s_l[warp][nt * 8 + rg + e] = l[nt][e];
          }
        }
      cons_sync();  // and every warp is done with the queries and masks, which O now overwrites
#pragma unroll
      for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = m[nt][e] == -INFINITY ? 0.f : ptx::ex2(m[nt][e] - row_max(nt * 8 + rg + e));
#pragma unroll
          for (int k = 0; k < kD / 16; ++k) {
            o[k][nt][e] *= f;
            o[k][nt][e + 2] *= f;
          }
        }
      // this lane's O of the unit's rows to or from a region
      auto put_o = [&](int region) {
#pragma unroll
        for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int rr = nt * 8 + rg + e;
            float* at = sO + (region * kRT + rr) * C::kOStride + kg;
            if (rr < rows) {
#pragma unroll
              for (int k = 0; k < kD / 16; ++k) {
                at[k * 16] = o[k][nt][e];
                at[k * 16 + 8] = o[k][nt][e + 2];
              }
            }
          }
      };
      auto add_o = [&](int region) {
#pragma unroll
        for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int rr = nt * 8 + rg + e;
            const float* at = sO + (region * kRT + rr) * C::kOStride + kg;
            if (rr < rows) {
#pragma unroll
              for (int k = 0; k < kD / 16; ++k) {
                o[k][nt][e] += at[k * 16];
                o[k][nt][e + 2] += at[k * 16 + 8];
              }
            }
          }
      };
#pragma unroll 1
      for (int half = C::kWarps / 2; half >= 1; half /= 2)
        for (int r = 0; r < half; r += C::kRegions) {
          const int up = warp - half - r, down = warp - r;
          if (up >= 0 && up < C::kRegions && warp < 2 * half) put_o(up);
          cons_sync();
          if (down >= 0 && down < C::kRegions && warp < half) add_o(down);
          cons_sync();
        }
      if (warp == 0) put_o(0);
      cons_sync();
      if constexpr (!kStream) {
        for (int rr = ct; rr < kRT; rr += C::kConsumers) s_ml[rr] = part_ml(rr);
        break;  // merged below, with the cluster's other parts
      }
      // ---- write the unit, or this CTA's part of it
      const auto [c0, c1] = unit_ctas(w);
      const int slot = unit_slot(blockIdx.x, sp.per, w.u0);
      const int quads = a.D / 4;
      for (int e = ct; e < rows * quads; e += C::kConsumers) {
        const int rr = e / quads, ch = e % quads, i = (r0 + rr) / a.G, g = (r0 + rr) % a.G;
        if (i >= n_act) continue;
        const float4 v = *reinterpret_cast<const float4*>(sO + rr * C::kOStride + ch * 4);
        const float2 ml = part_ml(rr);
        if (c1 <= c0) {
          const float inv = 1.f / ml.y;
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) +
                                    (((size_t)w.b * a.Hq + w.hk * a.G + g) * a.N + i) * a.D + ch * 4) =
              make_uint2(ptx::cvt_bf16x2(v.x * inv, v.y * inv), ptx::cvt_bf16x2(v.z * inv, v.w * inv));
        } else {
          __stcg(reinterpret_cast<float4*>(a.ws_o + ((size_t)slot * kRT + rr) * a.D + ch * 4), v);
          if (ch == 0) __stcg(a.ws_ml + (size_t)slot * kRT + rr, ml);
        }
      }
      if (c0 < c1) {
        __threadfence();
        cons_sync();
        if (ct == 0) {
          s_last = ptx::atom_add_acq_rel_gpu(&a.cnt[c0], 1u) == (unsigned)(c1 - c0);
          if (s_last) a.cnt[c0] = 0u;
          __threadfence();
        }
        cons_sync();
        if (s_last) {
          for (int e = ct; e < rows * quads; e += C::kConsumers) {
            const int rr = e / quads, ch = e % quads, i = (r0 + rr) / a.G, g = (r0 + rr) % a.G;
            if (i >= n_act) continue;
            // one pass in batches of independent loads, with a running maximum
            float M = -INFINITY, L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (long long cc = c0; cc <= c1; cc += kPmMerge) {
              float2 ml[kPmMerge];
              float4 v[kPmMerge];
#pragma unroll
              for (int k = 0; k < kPmMerge; ++k) {
                const size_t row = (size_t)unit_slot(min(cc + k, c1), sp.per, w.u0) * kRT + rr;
                ml[k] = __ldcg(&a.ws_ml[row]);
                v[k] = __ldcg(reinterpret_cast<const float4*>(a.ws_o + row * a.D + ch * 4));
                if (cc + k > c1) ml[k].x = -INFINITY;
              }
              float Mn = M;
#pragma unroll
              for (int k = 0; k < kPmMerge; ++k) Mn = fmaxf(Mn, ml[k].x);
              if (Mn == -INFINITY) continue;
              const float f0 = ptx::ex2(M - Mn);
              M = Mn;
              L *= f0;
              acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
#pragma unroll
              for (int k = 0; k < kPmMerge; ++k) {
                if (ml[k].x == -INFINITY) continue;
                const float f2 = ptx::ex2(ml[k].x - M);
                L = fmaf(f2, ml[k].y, L);
                acc.x = fmaf(f2, v[k].x, acc.x);
                acc.y = fmaf(f2, v[k].y, acc.y);
                acc.z = fmaf(f2, v[k].z, acc.z);
                acc.w = fmaf(f2, v[k].w, acc.w);
              }
            }
            const float inv = 1.f / L;
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) +
                                      (((size_t)w.b * a.Hq + w.hk * a.G + g) * a.N + i) * a.D + ch * 4) =
                make_uint2(ptx::cvt_bf16x2(acc.x * inv, acc.y * inv), ptx::cvt_bf16x2(acc.z * inv, acc.w * inv));
          }
        }
      }
    }
  }
  if constexpr (!kStream) {
    __syncwarp();
    ptx::cluster_sync();
    if (warp < C::kWarps) {
      const int quads = a.D / 4, items = rows * quads, share = (items + splits - 1) / splits;
      const uint32_t ml_local = ptx::smem_addr(s_ml), o_local = ptx::smem_addr(sm + C::kOffU);
      const int last = min(items, (int)(blockIdx.x + 1) * share);
      for (int e = blockIdx.x * share + threadIdx.x; e < last; e += C::kConsumers) {
        const int rr = e / quads, ch = e % quads, i = (r0 + rr) / a.G, g = (r0 + rr) % a.G;
        if (i >= n_act) continue;
        float2 ml[kPmMaxSplits];
        float4 v[kPmMaxSplits];
#pragma unroll
        for (int k = 0; k < kPmMaxSplits; ++k) {
          ml[k] = make_float2(-INFINITY, 0.f);
          if (k < splits) {
            ml[k] = ptx::ld_cluster_f32x2(ptx::map_cluster(ml_local, k) + rr * 8);
            v[k] = ptx::ld_cluster_f32x4(ptx::map_cluster(o_local, k) + (rr * C::kOStride + ch * 4) * 4);
          }
        }
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int k = 0; k < kPmMaxSplits; ++k) M = fmaxf(M, ml[k].x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kPmMaxSplits; ++k)
          if (ml[k].x != -INFINITY) {
            const float f = ptx::ex2(ml[k].x - M);
            L = fmaf(f, ml[k].y, L);
            acc.x = fmaf(f, v[k].x, acc.x);
            acc.y = fmaf(f, v[k].y, acc.y);
            acc.z = fmaf(f, v[k].z, acc.z);
            acc.w = fmaf(f, v[k].w, acc.w);
          }
        const float inv = 1.f / L;
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) +
                                  (((size_t)w.b * a.Hq + w.hk * a.G + g) * a.N + i) * a.D + ch * 4) =
            make_uint2(ptx::cvt_bf16x2(acc.x * inv, acc.y * inv), ptx::cvt_bf16x2(acc.z * inv, acc.w * inv));
      }
    }
    __syncwarp();
    ptx::cluster_sync();  // nobody leaves before its peers have read
  }
  __syncthreads();
  if (threadIdx.x == 0 && bars->abort) set_dev_status(a.dev_status, TV_DEV_TIMEOUT);
}

// ---- host side

struct PmPlan {
  int RT, row_tiles, splits;  // splits 0: persistent grid
  size_t rows, bytes;         // workspace of the persistent grid; clusters use none
};

static PmPlan pm_plan(int B, int Hq, int Hkv, int D, int N, int sms) {
  PmPlan p{};
  const int R = Hq / Hkv * N;
  p.RT = R <= 8 ? 8 : R <= 16 || D > 128 ? 16 : 32;  // O of 32 rows x 256 columns would not fit in registers
  p.row_tiles = (R + p.RT - 1) / p.RT;
  const long long units = (long long)B * Hkv * p.row_tiles;
  const bool few = units * 2 <= paged_device_sms() && B <= 65535 && units / B <= 65535;
  // units that run as clusters on the whole device do so on a share too, in fewer parts, unless the share
  // has fewer SMs than units: then its persistent grid has two slots a CTA, fewer than two a unit
  if (few) p.splits = (int)min((long long)kPmMaxSplits, sms / units);
  p.rows = 2 * (few ? (size_t)units : (size_t)kPagedMaxSms) * p.RT;
  p.bytes = kPagedCntBytes + p.rows * 8 + p.rows * D * 4;
  return p;
}

PagedWs paged_mma_ws(int B, int Hq, int Hkv, int D, int N, int sms) {
  const PmPlan p = pm_plan(B, Hq, Hkv, D, N, sms);
  return {p.bytes, p.splits ? 0 : p.bytes};
}

template <int kD, int kRT, int kCap, bool kStream>
static cudaError_t launch_pm(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const PmPlan& p,
                             cudaStream_t stream) {
  using C = PmCfg<kD, kRT>;
  const auto fn = paged_mma_kernel<kD, kRT, kCap, kStream>;
  const int wide = a.D == kD;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  if (kStream)
    return launch_pdl(fn, dim3((unsigned)a.sms), dim3(C::kThreads), C::kSmem, stream, nullptr, 0,
                      mk, mv, a, 0, p.row_tiles, wide);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  return launch_pdl(fn, dim3((unsigned)p.splits, (unsigned)(a.Hkv * p.row_tiles), (unsigned)a.B), dim3(C::kThreads),
                    C::kSmem, stream, attr, 1, mk, mv, a, p.splits, p.row_tiles, wide);
}

template <int kD, int kRT, int kCap>
static cudaError_t launch_pm_s(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const PmPlan& p,
                               cudaStream_t stream) {
  return p.splits ? launch_pm<kD, kRT, kCap, false>(mk, mv, a, p, stream)
                  : launch_pm<kD, kRT, kCap, true>(mk, mv, a, p, stream);
}

template <int kD, int kRT>
static cudaError_t launch_pm_c(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const PmPlan& p,
                               cudaStream_t stream) {
  switch (cap_mode(a.cap)) {
    case kLargeCap:
      return launch_pm_s<kD, kRT, kLargeCap>(mk, mv, a, p, stream);
    case kTanhCap:
      return launch_pm_s<kD, kRT, kTanhCap>(mk, mv, a, p, stream);
    default:
      return launch_pm_s<kD, kRT, kNoCap>(mk, mv, a, p, stream);
  }
}

template <int kD>
static cudaError_t launch_pm_d(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const PmPlan& p,
                               cudaStream_t stream) {
  if (p.RT == 8) return launch_pm_c<kD, 8>(mk, mv, a, p, stream);
  if constexpr (kD <= 128)
    if (p.RT == 32) return launch_pm_c<kD, 32>(mk, mv, a, p, stream);
  return launch_pm_c<kD, 16>(mk, mv, a, p, stream);
}

cudaError_t launch_paged_mma(PagedAttn a, char* ws, cudaStream_t stream) {
  const PmPlan p = pm_plan(a.B, a.Hq, a.Hkv, a.D, a.N, a.sms);
  if (!p.splits) {
    a.cnt = reinterpret_cast<unsigned*>(ws);
    a.ws_ml = reinterpret_cast<float2*>(ws + kPagedCntBytes);
    a.ws_o = reinterpret_cast<float*>(ws + kPagedCntBytes + p.rows * 8);
  }
  CUtensorMap mk, mv;
  if (!paged_kv_tmap(&mk, a.k, a) || !paged_kv_tmap(&mv, a.v, a)) return cudaErrorInvalidValue;
  if (a.D <= 64) return launch_pm_d<64>(mk, mv, a, p, stream);
  if (a.D <= 128) return launch_pm_d<128>(mk, mv, a, p, stream);
  return launch_pm_d<256>(mk, mv, a, p, stream);
}

}  // namespace tv
