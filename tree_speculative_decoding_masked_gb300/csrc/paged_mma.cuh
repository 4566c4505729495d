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
//
// Pages in 8 bits (kQ8, q8.cuh) are the same stream with half the bytes, in tiles of 128 keys, 32 a warp.
// K's codes go into e4m3 products as they are, with the queries' rows, times a power of two that brings the
// largest element to 2^7..2^8, as sums of two e4m3 numbers (off by half a step, 2^-10, or 2^-17 of the largest at most).  V's
// become fp16 numbers, which hold them exactly, in registers on the way: one conversion for two codes, where bf16,
// whose exponent is another, takes 4.5 instructions and more issue slots than the copies leave.  fp16's range is
// not that of the numbers, so V's scales stay out of it: with e the exponent of the value's block, P = 2^(z + e - m)
// and m is the running reference of z + e; the sum takes 2^-e times P, or, once an e is far from 0 (a block of zeros:
// q8_far), goes by z alone against a reference of its own, of each lane.  A weight keeps 11 bits while its product with 2^e
// is at least 2^-21 of the row's largest such product, fewer below, none below 2^-32.  A key's scale multiplies its scores, in fp32.  K's
// fragments need no transpose and any order of columns, if Q's have the same: a lane takes 16 columns of a key
// in one load.  Eight lanes take four such chunks of two keys, which the swizzle of 128-byte rows lays on
// different banks if the keys are four apart: so product row g is key g / 2 + 4 (g % 2) of its eight.  V's
// come by transposing loads of 16-bit pairs (two columns of a key), whose bytes are dealt to two product
// rows.  64 tokens over 8192 to 16384: 279 us, 5.7 TB/s (with values of zeros throughout 330); without the products the copies alone take 252, in boxes of
// 64-byte rows 260.  With K in fp16 too, 64 keys a tile, 16 a warp, and scales looked up for each key of a tile: 1900
// instructions for 64 keys and 390 us.  One token over 2048: 8.9 us; with a key a block 64 take 360.
#pragma once

#include "paged.cuh"
#include "q8.cuh"

namespace tv {

constexpr int kPmKeys = 64;
constexpr int kPmProducers = 4;
constexpr int kPmMaxSplits = 8;  // portable cluster size
constexpr int kPmMerge = 8;      // parts whose loads are in flight together
constexpr int kPmMinTiles = 2;   // tiles of a CTA's range: fewer only add parts to merge
// A unit's set-up and end count as 8 tiles, and cuts less than 8 from a unit's edge move to it
// (paged.cuh).  0 and 0 / 8 and 8: one token each of 64 sequences of 150 to 300 tokens 36.4 / 26.8 us,
// of 500 to 1000 50.8 / 46.4, of 8192 to 16384 465 / 461.
constexpr int kPmTol = 8, kPmFix = 8;  // in tiles of 64 keys
constexpr float kPmShift = 7.f;        // kQ8: P is held times 2^7

template <int kD, int kRT, bool kQ8>
struct PmCfg {
  static constexpr int kCols = kQ8 && kD > 64 ? 128 : 64;  // of a column block
  static constexpr int kDB = kD / kCols;
  static constexpr int kNT = kRT / 8;                   // row tiles of the products
  // consumers: two groups of four; one where O takes 128 registers a thread
  static constexpr int kWarps = kD == 256 || kD / 16 * kNT * 4 > 64 ? 4 : 8;
  static constexpr int kConsumers = kWarps * 32;
  static constexpr int kThreads = kConsumers + 32 * kPmProducers;
  static constexpr int kKeys = kQ8 ? 2 * kPmKeys : kPmKeys;  // of a tile
  static constexpr int kWarpKeys = kKeys / 4;
  static constexpr int kTol = kPmTol * kPmKeys / kKeys, kFix = kPmFix * kPmKeys / kKeys;
  static constexpr int kElt = kQ8 ? 1 : 2;
  static constexpr int kRow = kCols * kElt;             // bytes of a row in a block
  static constexpr int kBlock = 8 * kRow;
  static constexpr int kGroup = kDB * kBlock;           // 8 rows of a K or V tile: [column block][8][columns]
  static constexpr int kTile = kKeys / 8 * kGroup;
  static constexpr int kStages = kD == 64 ? 8 : kD == 128 ? (kRT <= 16 ? 6 : 5) : 3;  // of K and V
  // bytes: ldmatrix rows, or (kQ8) the 8-byte loads of four rows, on different banks
  static constexpr int kQStride = kD * 2 + (kQ8 ? 8 : 16);
  // K or V fragments loaded at once (kQ8: of V, as registers allow)
  static constexpr int kBatch = kQ8 && kNT > 2 ? 2 : (kQ8 && kNT > 1) || kD == 64 || kNT > 2 ? 4 : 8;
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
  static constexpr int kOffFar = kOffBar + 256;         // kQ8: sums of the threads' rows under far scales
  static constexpr int kSmem = kOffFar + (kQ8 ? kConsumers * 2 * kNT * 8 : 0) + 1024;
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

__device__ __forceinline__ void pm_mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void pm_mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pm_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Queries are held times 2^this, by the largest exponent field of their row: below 2^8.  A row that is not
// finite stays as it is.
__device__ __forceinline__ int pm_query_shift(int exponent) { return exponent == 255 ? 0 : min(127, 134 - exponent); }

// The next unit of this CTA: of its range, or the cluster's one unit, whether it has work or not.
// The producers and the consumers walk the same sequence of them.
template <int kRT, bool kStream, int kKeys>
__device__ __forceinline__ bool pm_next(const PagedAttn& a, UnitWalk& w, int splits) {
  if constexpr (kStream) return unit_next(a, w, kRT, kKeys);
  if (w.loaded == w.b) return false;
  bool bad;
  w.loaded = w.b;
  w.P = a.prefix_len[w.b];
  w.n = paged_rows(a, w.b, w.P, &bad);
  if (w.n == 0) w.P = 0;
  if (threadIdx.x == 0 && (bad || paged_cut(a, w.b, w.P, w.n))) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
  const int T_u = unit_tiles(a, w.P, w.n, w.rt, kRT, kKeys), part = blockIdx.x;
  w.t0 = (int)((long long)T_u * part / splits);
  w.t1 = (int)((long long)T_u * (part + 1) / splits);
  return true;
}

template <int kD, int kRT, int kCap, bool kStream, bool kQ8>
__global__ void __launch_bounds__(PmCfg<kD, kRT, kQ8>::kThreads, 1)
    paged_mma_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, PagedAttn a,
                     int splits, int row_tiles, int wide) {
  using C = PmCfg<kD, kRT, kQ8>;
  // kQ8: registers move from the producers to the consumers, 72 and 216 a thread of the launch's 168 (the launch bound's,
  // which ptxas takes for every kernel that moves any: 12 warps of 168 are 4 of 72 and 8 of 216).  They move once: a
  // second move would need each warpgroup's warps to meet before it, and producers never meet, so clusters, whose warps
  // share code at the end, move none.  Two row tiles spilled without (16 rows over 8192 to 16384, 64 sequences: 580
  // us, now 455; 8 rows 285, now 279).
  constexpr bool kShift = kQ8 && C::kWarps == 8 && kStream;
  ptx::griddep_launch_dependents();
  extern __shared__ unsigned char pm_raw[];
  unsigned char* sm = pm_raw + ((1024u - (ptx::smem_addr(pm_raw) & 1023u)) & 1023u);
  PmBars* bars = reinterpret_cast<PmBars*>(sm + C::kOffBar);
  volatile int* abort_flag = &bars->abort;
  __shared__ unsigned long long s_red[kPagedRed];
  __shared__ int s_lo[kRT], s_hi[kRT], s_first_pad, s_last;
  __shared__ float s_m[C::kWarps][kRT], s_l[C::kWarps][kRT];
  __shared__ __align__(8) float2 s_ml[kRT];
  __shared__ int s_qexp[kQ8 ? kRT : 1];  // a query row's largest exponent
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
    sp = paged_span(a, kRT, C::kKeys, kPmMinTiles, s_red, C::kTol, C::kFix);
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
    if constexpr (kShift) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // the boxes of a tile - (row piece, column block without 5-D boxes, K or V) - dealt to the
    // producer warps in turn; lane i of a warp looks up the page of its i-th box, read a tile
    // ahead and checked when it is used
    const int per_piece = 2 * (wide ? 1 : C::kDB);
    const int box_shift = min(a.page_shift, C::kDB == 1 || wide ? 6 : 3);
    const int boxes = (C::kKeys >> box_shift) * per_piece;
    const int mine = boxes / kPmProducers + (warp - C::kWarps < boxes % kPmProducers);
    const int box = lane * kPmProducers + warp - C::kWarps;  // this lane's
    const int pi = box / per_piece, part = box % per_piece;
    const uint32_t box_bytes = (uint32_t)(2 * kD * C::kElt / per_piece) << box_shift;
    // where it goes in a stage: K or V, 8-row group, column block
    const int off = (part & 1) * C::kTile + ((pi << box_shift) >> 3) * C::kGroup + (part >> 1) * C::kBlock;
    int issued = 0, counted = -1, active = 0;  // a sequence's active rows, once counted
    while (pm_next<kRT, kStream, C::kKeys>(a, w, splits)) {
      if (counted != w.b) {
        int pad = w.n;
        if (a.parent)
          for (int t = lane; t < w.n; t += 32)
            if (t > 0 && t < pad && a.parent[(size_t)w.b * a.N + t] == -1) pad = t;
        active = __reduce_min_sync(0xffffffffu, pad);
        counted = w.b;
      }
      const int unit = unit_rows(a, w.n, w.rt, kRT);
      const int lo = unit_lo(a, w.P, w.rt, kRT), tile0 = lo / C::kKeys;
      const int hi = min(w.P + active, w.P + (w.rt * kRT + unit - 1) / a.G + 1);
      const int32_t* table = a.table + (size_t)w.b * a.max_pages;
      // whether this lane's box in tile t holds a needed row, and its table entry
      auto needed = [&](int t) -> bool {
        const int j = (tile0 + t) * C::kKeys + (pi << box_shift);
        return t < w.t1 && lane < mine && j < hi && j + (1 << box_shift) > lo;
      };
      auto entry = [&](int t) -> int {
        return needed(t) ? table[((tile0 + t) * C::kKeys + (pi << box_shift)) >> a.page_shift] : 0;
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
          const int row = ((tile0 + t) * C::kKeys + (pi << box_shift)) & ((1 << a.page_shift) - 1);
          unsigned char* dst = sm + slot * 2 * C::kTile + off;
          const CUtensorMap* tm = (part & 1) ? &tmV : &tmK;
          if (C::kDB > 1 && wide)
            ptx::tma_load_5d(dst, tm, &bars->full[slot], 0, 0, 0, row >> 3, page * a.Hkv + w.hk);
          else
            ptx::tma_load_3d(dst, tm, &bars->full[slot], (part >> 1) * C::kCols, row, page * a.Hkv + w.hk);
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
    if constexpr (kShift) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
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
    while (pm_next<kRT, kStream, C::kKeys>(a, w, splits)) {
      rows = unit_rows(a, w.n, w.rt, kRT);
      r0 = w.rt * kRT;
      const int lo = unit_lo(a, w.P, w.rt, kRT), tile0 = lo / C::kKeys;
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
      if constexpr (kQ8) {
        if (ct < kRT) s_qexp[ct] = 1;
        cons_sync();
      }
      constexpr int kQChunks = (kRT * (kD / 8) + C::kConsumers - 1) / C::kConsumers;
      uint4 qraw[kQ8 ? kQChunks : 1];
      if constexpr (kQ8) {
#pragma unroll
        for (int k = 0; k < kQChunks; ++k) {
          const int e = k * C::kConsumers + ct;
          const int rr = e / (kD / 8), ch = e % (kD / 8), i = (r0 + rr) / a.G, g = (r0 + rr) % a.G;
          qraw[k] = make_uint4(0, 0, 0, 0);
          if (rr < rows && i < n_act && ch * 8 < a.D)
            qraw[k] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                                      (((size_t)w.b * a.Hq + w.hk * a.G + g) * a.N + i) * a.D + ch * 8);
          const uint32_t both = 0x7f807f80u;
          const uint32_t m = __vmaxu2(__vmaxu2(qraw[k].x & both, qraw[k].y & both),
                                      __vmaxu2(qraw[k].z & both, qraw[k].w & both));
          if (rr < kRT) atomicMax(&s_qexp[rr], (int)max(m >> 16, m & 0xffffu) >> 7);
        }
        cons_sync();
#pragma unroll
        for (int k = 0; k < kQChunks; ++k) {
          const int e = k * C::kConsumers + ct, rr = e / (kD / 8), ch = e % (kD / 8);
          if (rr >= kRT) break;
          const float f = q8_two(pm_query_shift(s_qexp[rr]));
          const uint32_t x[4] = {qraw[k].x, qraw[k].y, qraw[k].z, qraw[k].w};
          // row: the nearest e4m3 numbers, then the nearest to what they leave
          unsigned char* to = sQ + rr * C::kQStride + ch * 8;
          uint32_t hi[2], left[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float x0 = __uint_as_float(x[2 * u] << 16) * f, x1 = __uint_as_float(x[2 * u] & 0xffff0000u) * f;
            const float x2 = __uint_as_float(x[2 * u + 1] << 16) * f;
            const float x3 = __uint_as_float(x[2 * u + 1] & 0xffff0000u) * f;
            hi[u] = q8_code4(x0, x1, x2, x3);
            const float4 y = q8_numbers(hi[u], 1.f);
            left[u] = q8_code4(x0 - y.x, x1 - y.y, x2 - y.z, x3 - y.w);
          }
          *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(to + kD) = make_uint2(left[0], left[1]);
        }
      }
      for (int e = ct; !kQ8 && e < kRT * (kD / 8); e += C::kConsumers) {
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
      // kQ8: rows (lane >> 2) of a product, columns 64 j + 16 (lane & 3) + 8 s.. of step 2 j + s; the two parts are
      // kD bytes apart
      const unsigned char* qrow = sQ + (lane >> 2) * C::kQStride + (lane & 3) * 16;
      float row_f[C::kNT][2];
      if constexpr (kQ8) {
#pragma unroll
        for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) row_f[nt][e] = q8_two(-pm_query_shift(s_qexp[nt * 8 + rg + e]));
        if constexpr (C::kQRegs) {
#pragma unroll
          for (int k2 = 0; k2 < kD / 32; ++k2)
#pragma unroll
            for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const uint2 v =
                    *reinterpret_cast<const uint2*>(qrow + nt * 8 * C::kQStride + u * kD + (k2 >> 1) * 64 + (k2 & 1) * 8);
                qf[k2][nt][2 * u] = v.x, qf[k2][nt][2 * u + 1] = v.y;
              }
        }
      } else if constexpr (C::kQRegs) {
#pragma unroll
        for (int k2 = 0; k2 < kD / 32; ++k2)
#pragma unroll
          for (int nt = 0; nt < C::kNT; ++nt) pm_ldsm4(qf[k2][nt], qaddr + nt * 8 * C::kQStride + k2 * 64);
      }
      float o[kD / 16][C::kNT][4];
      float m[C::kNT][2], l[C::kNT][2];
      // kQ8: once a far scale has come, the sum of this lane and row is that of z alone, y times 2^x, in shared memory as few
      // calls have one.  To go back behind it, as paged_tc.cuh does, costs calls without one 1 to 3 % more
      bool far_on = false;
      auto far_sum = [&](int row) -> float2* { return reinterpret_cast<float2*>(sm + C::kOffFar) + row * C::kConsumers + ct; };
#pragma unroll
      for (int nt = 0; nt < C::kNT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int k = 0; k < kD / 16; ++k)
#pragma unroll
          for (int u = 0; u < 4; ++u) o[k][nt][u] = 0.f;
      }

      // kQ8: scales (K's byte, V's in bits 8..15).  Blocks of 16 keys or more: lane l looks up those of the warp's
      // keys 16 (l & 1).. of its turn l / 2 from here, for 16 turns at once, 16 turns ahead.  Shorter ones: of its
      // key l, two turns ahead.
      constexpr int kTurn = C::kWarps == 8 ? 2 : 1;
      const int32_t* table = a.table + (size_t)w.b * a.max_pages;
      const bool fine = kQ8 && a.block_shift < 4;
      auto scale_key = [&](int t) -> int {
        return fine ? (tile0 + t) * C::kKeys + wk * 32 + lane
                    : (tile0 + t + (lane >> 1) * kTurn) * C::kKeys + wk * 32 + (lane & 1) * 16;
      };
      auto scale_page = [&](int t) -> int {
        const int j = scale_key(t);
        return (fine ? t : t + (lane >> 1) * kTurn) < w.t1 && j + (fine ? 0 : 15) >= lo && j < hi ? table[j >> a.page_shift]
                                                                                                  : -1;
      };
      auto scale_bytes = [&](int t, int page) -> int {
        if (page < 0 || page >= a.num_pages) return 127 | 127 << 8;
        const size_t block = (((size_t)page * a.Hkv + w.hk) << (a.page_shift - a.block_shift)) +
                             ((scale_key(t) & ((1 << a.page_shift) - 1)) >> a.block_shift);
        return a.ks[block] | a.vs[block] << 8;
      };
      const int scale_step = fine ? kTurn : 16 * kTurn;
      int scales_now = 0, scales_next = 0, pages_next = -1, turn = 0;
      if constexpr (kQ8) {
        const int first = w.t0 + (C::kWarps == 8 && (it & 1) != group ? 1 : 0);
        const int p0 = scale_page(first), p1 = scale_page(first + scale_step);
        pages_next = scale_page(first + 2 * scale_step);
        scales_now = scale_bytes(first, p0);
        scales_next = scale_bytes(first + scale_step, p1);
      }
      for (int t = w.t0; t < w.t1; ++t, ++it) {
        if (C::kWarps == 8 && (it & 1) != group) continue;
        const int slot = it % C::kStages;
        int my_scales = 0;  // of this turn: lane 2 (turn & 15).., or every key's
        if constexpr (kQ8) {
          if (turn > 0 && (fine || turn % 16 == 0)) {
            scales_now = scales_next;
            scales_next = scale_bytes(t + scale_step, pages_next);
            pages_next = scale_page(t + 2 * scale_step);
          }
          my_scales = scales_now;
          ++turn;
        }
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars->full[slot], (it / C::kStages) & 1, abort_flag));
        if (!ok) continue;
        const int j0 = (tile0 + t) * C::kKeys + wk * C::kWarpKeys;  // this warp's keys
        unsigned char* sK = sm + slot * 2 * C::kTile + wk * (C::kWarpKeys / 8) * C::kGroup;
        unsigned char* sV = sK + C::kTile;
        if (j0 >= hi || j0 + C::kWarpKeys <= lo) {  // none of them
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bars->empty[slot]);
          continue;
        }
        const bool edge = j0 < lo || j0 + C::kWarpKeys > hi;
        if (edge) {
          // V rows that were not fetched or may hold anything, NaN included: zero
          constexpr int kRowChunks = C::kRow / 16;  // 16-byte chunks of a row in a column block
          for (int e = lane; e < C::kWarpKeys * C::kDB * kRowChunks; e += 32) {
            const int rr = e / (C::kDB * kRowChunks), rest = e % (C::kDB * kRowChunks);
            if (j0 + rr < lo || j0 + rr >= hi)
              *reinterpret_cast<uint4*>(sV + (rr >> 3) * C::kGroup + (rest / kRowChunks) * C::kBlock +
                                        (rr & 7) * C::kRow + rest % kRowChunks * 16) = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }
        // The slot goes back to the copies.  The fence orders this lane's reads and zeroes before their writes, which are
        // the async proxy's: without it the last ldmatrix of a tile read the next tile's values now and then
        auto free_slot = [&] {
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bars->empty[slot]);
        };
        if constexpr (kQ8) {
          // ---- 16 keys at a time; with one row tile both together, so that their latencies overlap
          auto key_of_row = [](int g) -> int { return C::kCols == 64 ? g : g >> 1 | (g & 1) << 2; };
          const int kk = key_of_row(kg);  // this lane's keys: kk, kk + 8
          constexpr int kSubs = C::kNT == 1 && kD <= 128 ? 2 : 1;
          const bool masked = j0 < full_lo || j0 + 32 > full_hi || edge;
#pragma unroll 1
          for (int sub0 = 0; sub0 < 2; sub0 += kSubs) {
            float s[kSubs][C::kNT][2][4];  // queries' two parts
            uint32_t pf[kSubs][C::kNT][2];
#pragma unroll
            for (int u = 0; u < kSubs; ++u) {
#pragma unroll
              for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[u][nt][0][x] = s[u][nt][1][x] = 0.f;
              const unsigned char* krow = sK + (sub0 + u) * 2 * C::kGroup + key_of_row(lane >> 2) * C::kRow;
#pragma unroll
              for (int j = 0; j < kD / 64; ++j) {
                const unsigned char* at =
                    C::kCols == 64 ? krow + (lane & 3) * 16
                                   : krow + (j >> 1) * C::kBlock + (((j & 1) * 4 + (lane & 3)) ^ key_of_row(lane >> 2)) * 16;
                const uint4 k0 = *reinterpret_cast<const uint4*>(at);
                const uint4 k1 = *reinterpret_cast<const uint4*>(at + C::kGroup);
#pragma unroll
                for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
                  for (int part = 0; part < 2; ++part) {
                    uint2 q0, q1;
                    if constexpr (C::kQRegs) {
                      q0 = make_uint2(qf[2 * j][nt][2 * part], qf[2 * j][nt][2 * part + 1]);
                      q1 = make_uint2(qf[2 * j + 1][nt][2 * part], qf[2 * j + 1][nt][2 * part + 1]);
                    } else {
                      const unsigned char* at = qrow + nt * 8 * C::kQStride + part * kD + j * 64;
                      q0 = *reinterpret_cast<const uint2*>(at);
                      q1 = *reinterpret_cast<const uint2*>(at + 8);
                    }
                    pm_mma_e4m3(s[u][nt][part], k0.x, k1.x, k0.y, k1.y, q0.x, q0.y);
                    pm_mma_e4m3(s[u][nt][part], k0.z, k1.z, k0.w, k1.w, q1.x, q1.y);
                  }
              }
            }
            // scores; those of a row's running reference count with the value's scale
            float val_e[kSubs][2], val_f[kSubs][2];  // e and 2^-e of keys kk, kk + 8
            bool grow = far_on;
#pragma unroll
            for (int u = 0; u < kSubs; ++u) {
              float key_f[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int from = fine ? (sub0 + u) * 16 + kk + 8 * e : ((turn - 1) & 15) * 2 + sub0 + u;
                const int both = __shfl_sync(0xffffffffu, my_scales, from);
                key_f[e] = __uint_as_float((uint32_t)(both & 255) << 23);
                val_e[u][e] = (float)((both >> 8) - 127);
                val_f[u][e] = __uint_as_float((uint32_t)max(1, 254 - (both >> 8)) << 23);
                grow |= q8_far(val_e[u][e]);
              }
#pragma unroll
              for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  float z = (s[u][nt][0][x] + s[u][nt][1][x]) * (key_f[x >> 1] * row_f[nt][x & 1]);
                  if constexpr (kCap == kTanhCap) z = soft_tanh(z * ck);
                  if constexpr (kCap == kLargeCap) z = capped_score(z * a.scale, a.cap, ck);
                  z = fmaf(z, c, val_e[u][x >> 1]);
                  if (masked) {
                    const int rr = nt * 8 + rg + (x & 1), j = j0 + (sub0 + u) * 16 + kk + (x >> 1) * 8;
                    bool vis = j >= s_lo[rr] && j < s_hi[rr];
                    if (!vis && a.parent && j >= w.P && j < hi)
                      vis = (s_vis[rr][(j - w.P) >> 5] >> ((j - w.P) & 31)) & 1u;
                    if (!vis) z = -INFINITY;
                  }
                  s[u][nt][0][x] = z;
                  grow |= z > m[nt][x & 1] + 8.f;
                }
            }
            if (__any_sync(0xffffffffu, grow)) {
              bool far = false;
#pragma unroll
              for (int u = 0; u < kSubs; ++u) far |= q8_far(val_e[u][0]) || q8_far(val_e[u][1]);
              if (__builtin_expect(__any_sync(0xffffffffu, far || far_on), 0)) {
                // few lines, as they sit among those of every turn: a loop over the rows, whose registers are selected
#pragma unroll 1
                for (int r = 0; r < 2 * C::kNT; ++r) {
                  float z[2 * kSubs], was_m = m[0][0] - kPmShift, was_l = l[0][0];
#pragma unroll
                  for (int k = 0; k < 2 * kSubs; ++k) z[k] = s[k >> 1][0][0][2 * (k & 1)];
#pragma unroll
                  for (int x = 1; x < 2 * C::kNT; ++x)
                    if (r == x) {
                      was_m = m[x >> 1][x & 1] - kPmShift, was_l = l[x >> 1][x & 1];
#pragma unroll
                      for (int k = 0; k < 2 * kSubs; ++k) z[k] = s[k >> 1][x >> 1][0][2 * (k & 1) + (x & 1)];
                    }
                  if (far_on) was_m = far_sum(r)->x, was_l = far_sum(r)->y;
                  float top = was_m;
#pragma unroll
                  for (int k = 0; k < 2 * kSubs; ++k) top = fmaxf(top, z[k] -= val_e[k >> 1][k & 1]);
                  const float base = top == -INFINITY ? 0.f : top;  // nothing seen yet: adds 0, or a NaN query's NaN
                  float sum = was_l * (top == was_m ? 1.f : ptx::ex2(was_m - top));
#pragma unroll
                  for (int k = 0; k < 2 * kSubs; ++k) sum += ptx::ex2(z[k] - base);
                  *far_sum(r) = make_float2(top, sum);
                }
                far_on = true;
              }
#pragma unroll
              for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float mx = fmaxf(s[0][nt][0][e], s[0][nt][0][e + 2]);
                  if (kSubs == 2) mx = fmaxf(mx, fmaxf(s[kSubs - 1][nt][0][e], s[kSubs - 1][nt][0][e + 2]));
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
#pragma unroll
            for (int nt = 0; nt < C::kNT; ++nt) {
              // at most 2^15
              const float b0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0] - kPmShift;
              const float b1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1] - kPmShift;
#pragma unroll
              for (int u = 0; u < kSubs; ++u) {
                const float e0 = ptx::ex2(s[u][nt][0][0] - b0), e1 = ptx::ex2(s[u][nt][0][1] - b1);
                const float e2 = ptx::ex2(s[u][nt][0][2] - b0), e3 = ptx::ex2(s[u][nt][0][3] - b1);
                l[nt][0] = fmaf(e0, val_f[u][0], fmaf(e2, val_f[u][1], l[nt][0]));
                l[nt][1] = fmaf(e1, val_f[u][0], fmaf(e3, val_f[u][1], l[nt][1]));
                pf[u][nt][0] = pm_transpose(pm_f16x2(e0, e1));
                pf[u][nt][1] = pm_transpose(pm_f16x2(e2, e3));
              }
            }
            // V^T: lane l names the key of row l & 7, of eight (l >> 3) & 1, and columns 16 (k + (l >> 4)).. of two steps
#pragma unroll
            for (int u = 0; u < kSubs; ++u) {
              const int vk = key_of_row(lane & 7);
              const uint32_t vaddr =
                  ptx::smem_addr(sV + (sub0 + u) * 2 * C::kGroup + ((lane >> 3) & 1) * C::kGroup + vk * C::kRow);
#pragma unroll
              for (int k0 = 0; k0 < kD / 16; k0 += C::kBatch) {
                uint32_t raw[C::kBatch / 2][4];
#pragma unroll
                for (int i = 0; i < C::kBatch / 2; ++i) {
                  const int k = k0 + 2 * i + (lane >> 4);
                  pm_ldsm4t(raw[i], C::kCols == 64 ? vaddr + (((k & 3) ^ (vk >> 1)) << 4)
                                                   : vaddr + (k >> 3) * C::kBlock + (((k & 7) ^ vk) << 4));
                }
#pragma unroll
                for (int i = 0; i < C::kBatch; ++i) {
                  // a word's bytes: columns 2g, 2g + 1 of key 2c, then of key 2c + 1; a product row is one column
                  uint32_t vf[4];
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const uint32_t word = raw[i >> 1][(i & 1) * 2 + x];
                    q8_half4(__byte_perm(word, 0, 0x3120), vf[2 * x], vf[2 * x + 1]);
                  }
#pragma unroll
                  for (int nt = 0; nt < C::kNT; ++nt) pm_mma_f16(o[k0 + i][nt], vf, pf[u][nt][0], pf[u][nt][1]);
                }
              }
            }
          }
          free_slot();
          continue;
        } else {
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
          free_slot();
        }
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
      if (kQ8 && __builtin_expect(far_on, 0)) {  // the sums' own references instead, and below O's
#pragma unroll 1
        for (int r = 0; r < 2 * C::kNT; ++r) {
          const float2 mine = *far_sum(r);
          float ref = mine.x;
#pragma unroll
          for (int x = 4; x < 32; x *= 2) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, x));
          float sum = mine.y * (mine.x == ref ? 1.f : ptx::ex2(mine.x - ref));
#pragma unroll
          for (int x = 4; x < 32; x *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          ref += (float)q8_norm(sum) + kPmShift;
          if (kg == 0) {
            s_m[warp][(r >> 1) * 8 + rg + (r & 1)] = sum == 0.f ? -INFINITY : ref;
            s_l[warp][(r >> 1) * 8 + rg + (r & 1)] = sum;
          }
        }
      }
      cons_sync();  // and every warp is done with the queries and masks, which O now overwrites
#pragma unroll
      for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float up = m[nt][e] - row_max(nt * 8 + rg + e);
          if (kQ8 && far_on) up *= 0.5f;  // half the exponent at a time: the whole may leave fp32's range
          const float f = m[nt][e] == -INFINITY ? 0.f : ptx::ex2(up);
#pragma unroll 1
          for (int twice = kQ8 && far_on; twice >= 0; --twice)
#pragma unroll
            for (int k = 0; k < kD / 16; ++k) {
              o[k][nt][e] *= f;
              o[k][nt][e + 2] *= f;
            }
        }
      // this lane's O of the unit's rows to or from a region: columns kg and kg + 8 of a step, or (kQ8) 2 kg and
      // 2 kg + 1
      constexpr int kPair = kQ8 ? 2 : 1, kNext = kQ8 ? 1 : 8;
      auto put_o = [&](int region) {
#pragma unroll
        for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int rr = nt * 8 + rg + e;
            float* at = sO + (region * kRT + rr) * C::kOStride + kg * kPair;
            if (rr < rows) {
#pragma unroll
              for (int k = 0; k < kD / 16; ++k) {
                at[k * 16] = o[k][nt][e];
                at[k * 16 + kNext] = o[k][nt][e + 2];
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
            const float* at = sO + (region * kRT + rr) * C::kOStride + kg * kPair;
            if (rr < rows) {
#pragma unroll
              for (int k = 0; k < kD / 16; ++k) {
                o[k][nt][e] += at[k * 16];
                o[k][nt][e + 2] += at[k * 16 + kNext];
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

template <int kD, int kRT, int kCap, bool kStream, bool kQ8>
static cudaError_t launch_pm(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const PmPlan& p,
                             cudaStream_t stream) {
  using C = PmCfg<kD, kRT, kQ8>;
  const auto fn = paged_mma_kernel<kD, kRT, kCap, kStream, kQ8>;
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

template <int kD, int kRT, int kCap, bool kQ8>
static cudaError_t launch_pm_s(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const PmPlan& p,
                               cudaStream_t stream) {
  return p.splits ? launch_pm<kD, kRT, kCap, false, kQ8>(mk, mv, a, p, stream)
                  : launch_pm<kD, kRT, kCap, true, kQ8>(mk, mv, a, p, stream);
}

template <int kD, int kRT, bool kQ8>
static cudaError_t launch_pm_c(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const PmPlan& p,
                               cudaStream_t stream) {
  switch (cap_mode(a.cap)) {
    case kLargeCap:
      return launch_pm_s<kD, kRT, kLargeCap, kQ8>(mk, mv, a, p, stream);
    case kTanhCap:
      return launch_pm_s<kD, kRT, kTanhCap, kQ8>(mk, mv, a, p, stream);
    default:
      return launch_pm_s<kD, kRT, kNoCap, kQ8>(mk, mv, a, p, stream);
  }
}

template <int kD, bool kQ8>
static cudaError_t launch_pm_d(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const PmPlan& p,
                               cudaStream_t stream) {
  if (p.RT == 8) return launch_pm_c<kD, 8, kQ8>(mk, mv, a, p, stream);
  if constexpr (kD <= 128)
    if (p.RT == 32) return launch_pm_c<kD, 32, kQ8>(mk, mv, a, p, stream);
  return launch_pm_c<kD, 16, kQ8>(mk, mv, a, p, stream);
}

// launch_pm_d<256, true>, a file of its own to compile
cudaError_t launch_pm_q8_wide(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, const PmPlan& p,
                              cudaStream_t stream);

template <bool kQ8>
static cudaError_t launch_pm_all(PagedAttn a, char* ws, cudaStream_t stream) {
  const PmPlan p = pm_plan(a.B, a.Hq, a.Hkv, a.D, a.N, a.sms);
  if (!p.splits) {
    a.cnt = reinterpret_cast<unsigned*>(ws);
    a.ws_ml = reinterpret_cast<float2*>(ws + kPagedCntBytes);
    a.ws_o = reinterpret_cast<float*>(ws + kPagedCntBytes + p.rows * 8);
  }
  CUtensorMap mk, mv;
  const bool made = kQ8 ? paged_q8_tmap(&mk, a.k, a, a.D <= 64 ? kQ8Plain : kQ8Rows128) &&
                              paged_q8_tmap(&mv, a.v, a, a.D <= 64 ? kQ8Swizzled : kQ8Rows128)
                        : paged_kv_tmap(&mk, a.k, a) && paged_kv_tmap(&mv, a.v, a);
  if (!made) return cudaErrorInvalidValue;
  if (a.D <= 64) return launch_pm_d<64, kQ8>(mk, mv, a, p, stream);
  if (a.D <= 128) return launch_pm_d<128, kQ8>(mk, mv, a, p, stream);
  if constexpr (kQ8)
    return launch_pm_q8_wide(mk, mv, a, p, stream);
  else
    return launch_pm_d<256, false>(mk, mv, a, p, stream);
}

}  // namespace tv
