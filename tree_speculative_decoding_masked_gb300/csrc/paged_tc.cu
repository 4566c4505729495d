// Attention of new rows over a paged KV cache on the 5th-generation tensor cores (tcgen05,
// TMEM, TMA), for chunks and trees whose rows fill row tiles.
//
//   S = Q K^T,  P = 2^(c S - m) over the visible keys,  O += P V,  out = O / sum P
//
// with the softmax's maximum and sum in 32 bits and P rounded to bf16 for the second product
// (2^-8 of each weight, the tensor core's input type).  One CTA owns two 128-row tiles A and
// B of one (sequence, KV head) - the G query heads of NT = 128 / G nodes each - and streams a
// range of 64-key tiles once for both, so a page fetched from L2 serves 256 rows.
//
// Pages: a tile is fetched in boxes of min(page_size, 64) rows, each by a lane of the producer
// warp from the page that its own table entry names, read ahead.  At D = 128 a box is 5-D
// (64 columns, 8 rows, 2 column halves, row groups of 8): both halves come in one copy, laid
// out as 8-row groups of [half][8 rows][128 bytes], whose group stride of 2 KB the products'
// descriptors carry.  Boxes of 64 columns each would be twice as many, and at 16-row pages
// the copies' issue, not their bytes, set the pace (590 us for eight 128-node trees over
// 32768 tokens against 428 at 64-row pages).  Boxes that hold no needed row are not fetched
// and their table entries not used.  V rows outside the needed range (the tail of a
// sequence's last page, rows behind the window) may hold anything, NaN included, which a
// zero weight would not remove: the PV issuer's warp zeroes them in shared memory first.
//
// Warps: 0 producer (V a tile behind K), 1 S issuer of tile A (loads its Q) and TMEM owner,
// 2-9 softmax (four per tile, one row a thread), 10 PV issuer, 11 S issuer of tile B.
// TMEM columns: S_A[0] 0.., S_A[1] 64.., S_B[0] 128.., S_B[1] 192.., O_A 256.., O_B 384...
// P_X (bf16, 32 columns) overwrites the first half of its own S buffer.
//
// Two schedules.  Where clusters of two or more CTAs hold all row tiles (or pairs) at once, each
// one's keys are cut into equal parts that run as one thread-block cluster and merge behind its
// barrier; a CTA with one tile has half the partial rows to park and merge, which costs a
// short range more than K and V read twice.  Otherwise a persistent grid of one CTA per SM divides
// all pairs' 64-key steps equally (paged.cuh), which keeps ragged batches and causal triangles
// balanced; a pair cut between CTAs is merged through the workspace, in CTA order, by the CTA that
// finishes last.  There the pieces follow one another without a stop: the producer finds each
// and posts it, keeps the rings filled across pieces, and Q and the first scores of the next
// are there when the softmax warps have written a piece out.  With a stop and a fresh set-up
// at each piece, and every warp finding it for itself, 16 chunks of 512 rows over 1000 to 2000
// tokens took 264 us, now 238; two of 2048 rows over 3000 to 6000 326, now 310.
#include <atomic>

#include "paged.cuh"

namespace tv {

constexpr int kPtRows = 128;
constexpr int kPtKeys = 64;
constexpr int kPtSlots = 4;      // K ring and V ring depth
constexpr int kPtThreads = 384;  // 12 warps
constexpr int kPtPieces = 4;     // pieces known ahead
constexpr int kPtMaxSplits = 8;  // portable cluster size
// A unit's set-up and end count as 8 steps, and cuts less than 12 from a unit's edge move to it
// (paged.cuh).  0 and 0 / 12 and 0 / 12 and 8: nine causal chunks of 1510 to 1758 rows on empty caches
// 72.5 / 61.3 / 56.2 us, one of 2048 rows 81.5 / 68.2 / 57.9, 64 trees of 16 nodes over 1000 tokens
// 92.7 / 77.0 / 77.4.
constexpr int kPtTol = 12;
constexpr int kPtFix = 8;
constexpr float kPtRescaleLog2 = 8.f;
constexpr float kPtRescaleSum = 256.f;

template <int D>
struct PtCfg {
  static constexpr int kDB = D / 64;
  static constexpr int kQBlock = kPtRows * 128;      // bytes per 64-column block of one Q tile
  static constexpr int kQTile = kDB * kQBlock;
  static constexpr int kGroup = kDB * 1024;          // a K or V tile's 8-row group: [column block][8][128 bytes]
  static constexpr int kTileBytes = kPtKeys / 8 * kGroup;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + 2 * kQTile;
  static constexpr int kOffV = kOffK + kPtSlots * kTileBytes;
  static constexpr int kOffPar = kOffV + kPtSlots * kTileBytes;
  static constexpr int kOffBar = kOffPar + kMaxNodes * 4;
  static constexpr int kSmemAlloc = kOffBar + 512 + 1024;  // slack for 1024-byte alignment
  static constexpr uint32_t kColO = 256;
  static_assert(kSmemAlloc + 8192 <= 232448, "shared memory per CTA");  // 8192: paged_span's and the pieces'
};

struct PtBars {
  uint64_t q_full[2];
  uint64_t k_full[kPtSlots];
  uint64_t k_empty[kPtSlots];
  uint64_t v_full[kPtSlots];
  uint64_t v_empty[kPtSlots];
  uint64_t s_full[2][2];
  uint64_t p_full[2][2];
  uint64_t pv_done[2][2];
  uint64_t o_done;
  uint64_t s_done[2];
  uint64_t o_free[2];  // tile x's warps have read O
  uint64_t rows_met;   // the softmax warps meet
  uint64_t piece_full[kPtPieces];
  uint64_t piece_empty[kPtPieces];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(PtBars) <= 512);

// One piece of work, a range of a unit's key tiles: what the producer finds and every warp goes by.
struct PtPiece {
  int b, hk, rt, P, n;  // unit; the sequence's committed and new rows
  int t0, t1;           // of the unit's tiles, those to take
  int c0, c1;           // CTAs that share the unit, c1 <= c0: it is this CTA's alone
  int slot0;            // where CTA c0 parks its part (the others: 2 c)
  int slot;             // and this one
  int more;             // 0: there is none
};
struct PtArgs {
  int NT;      // nodes per row tile
  int tiles;   // row tiles per unit: 2, or 1 (cluster schedule of few tiles)
  int MP;      // units per (sequence, KV head)
  int splits;  // cluster schedule: parts of a pair's keys
  int wide;    // K and V boxes span both column blocks (5-D maps)
};

__device__ __forceinline__ float pt_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float pt_max64(const float (&sv)[64]) {
  float c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) c[k] = fmaxf(sv[2 * k], sv[2 * k + 1]);
#pragma unroll
  for (int j = 8; j < 64; j += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = pt_max3(c[k], sv[j + 2 * k], sv[j + 2 * k + 1]);
  return fmaxf(fmaxf(c[0], c[1]), fmaxf(c[2], c[3]));
}
// P = 2^(s c - m) as bf16 pairs; returns the sum of the unrounded values.  m = -inf: no key
// has been visible yet and every s is -inf, so P is 0 with any finite offset.
__device__ __forceinline__ float pt_exp64(const float (&sv)[64], float c, float m, uint32_t (&pw)[32]) {
  const float nm = m == -INFINITY ? 0.f : -m;
  const float2 cc = make_float2(c, c), nm2 = make_float2(nm, nm);
  float2 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const float2 t = __ffma2_rn(make_float2(sv[2 * k], sv[2 * k + 1]), cc, nm2);
    const float e0 = ptx::ex2(t.x), e1 = ptx::ex2(t.y);
    acc[k & 3] = __fadd2_rn(acc[k & 3], make_float2(e0, e1));
    pw[k] = ptx::cvt_bf16x2(e0, e1);
  }
  const float2 s2 = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
  return s2.x + s2.y;
}
// v[x] of two by selection: a runtime index would put them in local memory, which every step's
// waits would then read again (0.1 us a step)
template <typename T>
__device__ __forceinline__ T pt_of(const T (&v)[2], int x) {
  return x ? v[1] : v[0];
}
// bits [lo, hi) of a 64-bit word
__device__ __forceinline__ uint64_t pt_bits(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 64);
  if (hi <= lo) return 0ull;
  const uint64_t up = hi == 64 ? ~0ull : (1ull << hi) - 1ull;
  return up & ~((1ull << lo) - 1ull);
}

// S of one row tile (K = D in steps of 16) as one asm block: an issuing thread shares its
// sub-partition with softmax warps, and fewer instructions per product issue the short
// (N = 64) products sooner.  bd steps 32 bytes inside a 128-byte row, 1 KB to the second
// column block.
__device__ __forceinline__ void pt_s_product(uint32_t d, const uint64_t (&ad)[8], uint64_t bd, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b32 z;\n\tmov.b32 z, 0;\n\tsetp.ne.b32 p0, z, 0;\n\tsetp.eq.b32 p1, z, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %9, %17, p0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %10, %17, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %11, %17, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %12, %17, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %5, %13, %17, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %6, %14, %17, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %7, %15, %17, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %8, %16, %17, p1;\n\t}" ::"r"(d),
      "l"(ad[0]), "l"(ad[1]), "l"(ad[2]), "l"(ad[3]), "l"(ad[4]), "l"(ad[5]), "l"(ad[6]), "l"(ad[7]), "l"(bd),
      "l"(bd + 2), "l"(bd + 4), "l"(bd + 6), "l"(bd + 64), "l"(bd + 66), "l"(bd + 68), "l"(bd + 70), "r"(idesc)
      : "memory");
}
__device__ __forceinline__ void pt_s_product(uint32_t d, const uint64_t (&ad)[4], uint64_t bd, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) ptx::mma_bf16_ss(d, ad[kk], bd + kk * 2, idesc, kk > 0 ? 1u : 0u);
}
// O += P V of 64 keys: P from TMEM (8 columns per 16 keys), V rows 16 apart (`step` 16-byte units)
__device__ __forceinline__ void pt_pv_product(uint32_t d, uint32_t p, uint64_t vd, uint32_t step, uint32_t idesc,
                                              uint32_t acc0) {
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b32 z;\n\tmov.b32 z, 0;\n\tsetp.ne.b32 p0, %10, 0;\n\tsetp.eq.b32 p1, z, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %5, %9, p0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %6, %9, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %7, %9, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], %8, %9, p1;\n\t}" ::"r"(d),
      "r"(p), "r"(p + 8), "r"(p + 16), "r"(p + 24), "l"(vd), "l"(vd + step), "l"(vd + 2 * step), "l"(vd + 3 * step),
      "r"(idesc), "r"(acc0)
      : "memory");
}

// Wait for this piece's own copies or products even when another wait has run out.
__device__ __forceinline__ void pt_drain(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  int quiet = 0;
  if (!ptx::mbar_wait(bar, parity, &quiet)) *abort_flag = 1;
}

__device__ __forceinline__ void pt_bars_init(PtBars* bars) {
  ptx::mbar_init(&bars->q_full[0], 1);
  ptx::mbar_init(&bars->q_full[1], 1);
  ptx::mbar_init(&bars->rows_met, 8);
  for (int s = 0; s < kPtPieces; ++s) {
    ptx::mbar_init(&bars->piece_full[s], 1);
    ptx::mbar_init(&bars->piece_empty[s], kPtThreads / 32 - 1);
  }
  for (int s = 0; s < kPtSlots; ++s) {
    ptx::mbar_init(&bars->k_full[s], 1);
    ptx::mbar_init(&bars->k_empty[s], 2);  // both S issuers
    ptx::mbar_init(&bars->v_full[s], 1);
    ptx::mbar_init(&bars->v_empty[s], 1);
  }
  for (int x = 0; x < 2; ++x)
    for (int u = 0; u < 2; ++u) {
      ptx::mbar_init(&bars->s_full[x][u], 1);
      ptx::mbar_init(&bars->p_full[x][u], 4);
      ptx::mbar_init(&bars->pv_done[x][u], 1);
    }
  ptx::mbar_init(&bars->o_done, 1);
  ptx::mbar_init(&bars->s_done[0], 1);
  ptx::mbar_init(&bars->s_done[1], 1);
  ptx::mbar_init(&bars->o_free[0], 4);
  ptx::mbar_init(&bars->o_free[1], 4);
  ptx::fence_mbar_init();
}

template <int D, int kCap, bool kStream>
__global__ void __launch_bounds__(kPtThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, PagedAttn a, PtArgs pa) {
  ptx::griddep_launch_dependents();
  using C = PtCfg<D>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t mis = ptx::smem_addr(smem_raw) & 1023u;
  unsigned char* sm = smem_raw + ((1024u - mis) & 1023u);
  unsigned char* sQ = sm + C::kOffQ;
  unsigned char* sK = sm + C::kOffK;
  unsigned char* sV = sm + C::kOffV;
  int* s_par = reinterpret_cast<int*>(sm + C::kOffPar);
  PtBars* bars = reinterpret_cast<PtBars*>(sm + C::kOffBar);
  volatile int* abort_flag = &bars->abort;
  __shared__ unsigned long long s_red[kPagedRed];
  __shared__ int s_last;
  __shared__ PtPiece s_piece[kPtPieces];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int NT = pa.NT, rows_used = a.G * NT, RT = pa.tiles * rows_used;
  if (warp == 1) {
    ptx::tmem_alloc(&bars->tmem_base, 512);
    ptx::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&tmQ);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
    bars->abort = 0;
    pt_bars_init(bars);
  }
  // the Q rows that no box fills
  for (int r = rows_used + threadIdx.x; r < 2 * kPtRows; r += kPtThreads) {
    const int x = r >= kPtRows ? 1 : 0, rr = r - x * kPtRows;
    if (rr < rows_used) continue;
    for (int db = 0; db < C::kDB; ++db) {
      uint4* row = reinterpret_cast<uint4*>(sQ + x * C::kQTile + db * C::kQBlock + rr * 128);
#pragma unroll
      for (int k = 0; k < 8; ++k) row[k] = make_uint4(0, 0, 0, 0);
    }
  }
  ptx::fence_proxy_async_smem();
  // shared memory, TMEM and parameters only so far: this overlaps the previous kernel's tail
  ptx::griddep_wait();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // ---- this CTA's pieces
  UnitWalk w{};  // the producer's
  const size_t cta = ((size_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;  // cluster schedule
  if constexpr (kStream) {
    const PagedSpan sp = paged_span<true>(a, RT, kPtKeys, 1, s_red, kPtTol, kPtFix);
    w = unit_walk(sp);
  }
  // the softmax warps meet.  Between pieces by an mbarrier: a hardware barrier would hang if the wait for a
  // piece ran out in some of them only
  unsigned met = 0;
  auto softmax_sync = [&] {
    if constexpr (kStream) {
      int quiet = 0;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars->rows_met);
      if (!ptx::mbar_wait(&bars->rows_met, met & 1, &quiet)) *abort_flag = 1;
      ++met;
      __syncwarp();
    } else {
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
  };
  int loaded_b = -1, n_act = 0;
  // tiles, and tiles with rows of A and B, of the pieces before this one, and how many those were: what
  // the rings' slots and the barriers' phases go by.  Every role counts them alike.
  unsigned kt = 0, done_x[2] = {0, 0}, pieces = 0;
  unsigned k_issued = 0, v_issued = 0;  // the producer's copies
  unsigned q_loads = 0;                 // an S issuer's
  bool ok = true;                       // no wait of this role has run out
  auto drain = [&] {  // the producer: no copy is in flight when the CTA ends
    for (unsigned s = 0; s < kPtSlots; ++s) {
      if (s < k_issued) pt_drain(&bars->k_full[s], ((k_issued - 1 - s) / kPtSlots) & 1, abort_flag);
      if (s < v_issued) pt_drain(&bars->v_full[s], ((v_issued - 1 - s) / kPtSlots) & 1, abort_flag);
    }
  };
  for (unsigned np = 0;; ++np) {
    PtPiece pc;
    if constexpr (kStream) {
      // the producer runs ahead of the others: it finds the pieces and posts them
      const int ps = np % kPtPieces;
      int quiet = 0;  // pieces come after an abort too, so that each cut unit's parts are counted
      if (warp == 0) {
        pc.more = unit_next(a, w, RT, kPtKeys);
        pc.b = w.b, pc.hk = w.hk, pc.rt = w.rt, pc.P = w.P, pc.n = w.n, pc.t0 = w.t0, pc.t1 = w.t1;
        const UnitCtas by = unit_ctas(w);
        pc.c0 = (int)by.c0, pc.c1 = (int)by.c1;
        pc.slot0 = unit_slot(by.c0, w.per, w.u0), pc.slot = unit_slot(blockIdx.x, w.per, w.u0);
        bool got = true;
        if (np >= kPtPieces)
          got = ptx::mbar_wait_limit(&bars->piece_empty[ps], (np / kPtPieces - 1) & 1, &quiet, 8 * TV_WAIT_NS);
        if (!__all_sync(0xffffffffu, got)) {
          *abort_flag = 1;
          break;
        }
        if (lane == 0) {
          s_piece[ps] = pc;
          ptx::mbar_arrive(&bars->piece_full[ps]);
        }
        __syncwarp();
      } else {
        const bool got =
            ptx::mbar_wait_limit(&bars->piece_full[ps], (np / kPtPieces) & 1, &quiet, 8 * TV_WAIT_NS);
        if (!__all_sync(0xffffffffu, got)) {
          *abort_flag = 1;
          break;
        }
        const PtPiece& at = s_piece[ps];
        pc.b = at.b, pc.hk = at.hk, pc.rt = at.rt, pc.P = at.P, pc.n = at.n, pc.t0 = at.t0, pc.t1 = at.t1;
        pc.more = at.more;
      }
      if (!pc.more) break;
    } else {
      pc.b = blockIdx.z, pc.hk = blockIdx.y, pc.rt = pa.MP - 1 - (int)blockIdx.x / pa.splits;
    }
    const int b = pc.b, hk = pc.hk, mp = pc.rt;
    if (b != loaded_b) {
      // Tree rows count up to the first padding row (a tree with rows behind it is bad).  Every warp
      // counts for itself, and the softmax warps check and keep the parents.  The first reads
      // run beside those of the lengths.
      const int32_t* par = a.parent ? a.parent + (size_t)b * a.N : nullptr;
      const int st = (int)threadIdx.x - 64;
      const bool rows_warp = warp >= 2 && warp < 10;
      int first[4], p_first = -1, p_before = -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) first[k] = par && k * 32 + lane < a.N ? par[k * 32 + lane] : -1;
      if (par && rows_warp && st < a.N) {
        p_first = par[st];
        if (st > 0) p_before = par[st - 1];
      }
      if constexpr (!kStream) {
        bool bad = false;
        pc.P = a.prefix_len[b];
        pc.n = paged_rows(a, b, pc.P, &bad);
        if (pc.n == 0) pc.P = 0;
        if (threadIdx.x == 0 && (bad || paged_cut(a, b, pc.P, pc.n))) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
      }
      const int n = pc.n;
      n_act = n;
      if (par && n > 0) {
        int count = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = k * 32 + lane;
          count += t > 0 && t < n && first[k] != -1;
        }
        for (int t = 128 + lane; t < n; t += 32) count += par[t] != -1;
        n_act = 1 + __reduce_add_sync(0xffffffffu, count);
        if (rows_warp) {
          if (loaded_b >= 0) softmax_sync();  // the piece before's rows have read s_par
          for (int t = st; t < n; t += 256) {
            const int p = t == st ? p_first : par[t];
            const bool prev_pad = t >= 2 && (t == st ? p_before : par[t - 1]) == -1;
            const bool fits = t == 0 ? p == -1 : (p == -1 || (p >= 0 && p < t && !prev_pad));
            if (!fits) set_dev_status(a.dev_status, TV_DEV_BAD_TREE);
            s_par[t] = fits ? p : -1;
          }
          softmax_sync();
        }
      }
      loaded_b = b;
    }
    const int P = pc.P, n = pc.n;
    const int lo = unit_lo(a, P, mp, RT);
    int split = 0;
    if constexpr (!kStream) {
      const int T_u = unit_tiles(a, P, n, mp, RT, kPtKeys);
      split = blockIdx.x % pa.splits;
      pc.t0 = (int)((long long)T_u * split / pa.splits);
      pc.t1 = (int)((long long)T_u * (split + 1) / pa.splits);
    }
    const int t_begin = lo / kPtKeys + pc.t0;  // this piece's key tiles
    const int nt_all = pc.t1 - pc.t0;
    const int key_end = P + n_act;  // rows from here on, and before lo, may hold anything
    int i0[2], ntx[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      i0[x] = (pa.tiles * mp + x) * NT;
      const int hi = x < pa.tiles && i0[x] < n_act ? P + min(n_act, i0[x] + NT) : 0;
      ntx[x] = max(0, min(nt_all, (hi + kPtKeys - 1) / kPtKeys - t_begin));
    }
    const int nt = max(ntx[0], ntx[1]);

    float m_run = -INFINITY, l_run = 0.f;
    bool have_o = false;
    if (warp == 0) {
      // ---------------------------------------------------------------- producer
      // lane: row piece pi of a tile (and, without 5-D boxes, its column block db)
      const int per_piece = pa.wide ? 1 : C::kDB;
      const int box_shift = min(a.page_shift, C::kDB == 1 || pa.wide ? 6 : 3);
      const int db = lane % per_piece, pi = lane / per_piece;
      const bool in_tile = (pi << box_shift) < kPtKeys;
      const uint32_t box_bytes = (uint32_t)(128 * C::kDB / per_piece) << box_shift;
      const int32_t* table = a.table + (size_t)b * a.max_pages;
      // whether this lane's box in tile t holds a needed row, and its table entry (read two tiles
      // ahead, checked when it is used)
      auto needed = [&](int t) -> bool {
        const int j = (t_begin + t) * kPtKeys + (pi << box_shift);
        return t < nt && in_tile && j < key_end && j + (1 << box_shift) > lo;
      };
      auto entry = [&](int t) -> int {
        return needed(t) ? table[((t_begin + t) * kPtKeys + (pi << box_shift)) >> a.page_shift] : 0;
      };
      auto checked = [&](int t, int page) -> int {
        if (!needed(t)) return -1;
        if (page >= 0 && page < a.num_pages) return page;
        set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
        return -1;
      };
      int raw0 = entry(0), raw1 = entry(1), before = -1;
      // this lane's box of tile t into its ring slot; false after an abort
      auto fetch = [&](unsigned char* ring, const CUtensorMap* tm, uint64_t* full, uint64_t* empty, int t,
                       int pg) -> bool {
        const unsigned gt = kt + t;
        const int slot = gt % kPtSlots;
        bool got = true;
        if (gt >= kPtSlots) got = ptx::mbar_wait(&empty[slot], ((gt / kPtSlots) - 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, got)) return false;
        const uint32_t boxes = __ballot_sync(0xffffffffu, pg >= 0);
        if (lane == 0) ptx::mbar_arrive_expect_tx(&full[slot], __popc(boxes) * box_bytes);
        __syncwarp();
        if (pg >= 0) {
          const int row = ((t_begin + t) * kPtKeys + (pi << box_shift)) & ((1 << a.page_shift) - 1);
          unsigned char* dst = ring + slot * C::kTileBytes + ((pi << box_shift) >> 3) * C::kGroup + db * 1024;
          if (C::kDB > 1 && pa.wide)
            ptx::tma_load_5d(dst, tm, &full[slot], 0, 0, 0, row >> 3, pg * a.Hkv + hk);
          else
            ptx::tma_load_3d(dst, tm, &full[slot], db * 64, row, pg * a.Hkv + hk);
        }
        return true;
      };
      for (int t = 0; ok && t <= nt && nt > 0; ++t) {
        const int page = checked(t, raw0);
        raw0 = raw1;
        raw1 = entry(t + 2);
        if (t < nt) {
          if (!(ok = fetch(sK, &tmK, bars->k_full, bars->k_empty, t, page))) break;
          k_issued = kt + t + 1;
        }
        if (t > 0) {
          if (!(ok = fetch(sV, &tmV, bars->v_full, bars->v_empty, t - 1, before))) break;
          v_issued = kt + t;
        }
        before = page;
      }
      if (!kStream && lane == 0) drain();
    } else if (warp == 1 || warp == 11) {
      // ---------------------------------------------------------------- S issuer of tile x
      const int x = warp == 1 ? 0 : 1;
      if (lane == 0) {
        const int ntm = pt_of(ntx, x);
        const unsigned dx = pt_of(done_x, x);
        if (ntm > 0) {
          ptx::mbar_arrive_expect_tx(&bars->q_full[x], (uint32_t)(rows_used * 128 * C::kDB));
          for (int g = 0; g < a.G; ++g)
            for (int d = 0; d < C::kDB; ++d)
              ptx::tma_load_3d(sQ + x * C::kQTile + d * C::kQBlock + g * NT * 128, &tmQ, &bars->q_full[x], d * 64,
                               pt_of(i0, x), b * a.Hq + hk * a.G + g);
          pt_drain(&bars->q_full[x], q_loads++ & 1, abort_flag);
        }
        if (nt > 0) {
          constexpr uint32_t idS = ptx::idesc_bf16(kPtRows, kPtKeys, false, false);
          const uint32_t qaddr = ptx::smem_addr(sQ + x * C::kQTile);
          uint64_t adq[D / 16];
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            adq[kk] = ptx::sdesc_sw128(qaddr + (kk >> 2) * C::kQBlock + (kk & 3) * 32, 16, 1024);
          for (int t = 0; ok && t < nt; ++t) {
            const int ks = (kt + t) % kPtSlots;
            if (!(ok = ptx::mbar_wait(&bars->k_full[ks], ((kt + t) / kPtSlots) & 1, abort_flag))) break;
            if (t < ntm) {
              // S_X(t) overwrites P_X of two tiles before in this buffer
              const unsigned tx = dx + t;
              const int buf = tx & 1;
              if (tx >= 2 && !(ok = ptx::mbar_wait(&bars->pv_done[x][buf], ((tx - 2) >> 1) & 1, abort_flag))) break;
              ptx::tc_fence_after();
              pt_s_product(tmem + x * kPtRows + buf * kPtKeys, adq,
                           ptx::sdesc_sw128(ptx::smem_addr(sK + ks * C::kTileBytes), 16, C::kGroup), idS);
              ptx::mma_commit(&bars->s_full[x][buf]);
            }
            ptx::mma_commit(&bars->k_empty[ks]);
          }
          // Q's place is free again behind its products
          ptx::mma_commit(&bars->s_done[x]);
          pt_drain(&bars->s_done[x], pieces & 1, abort_flag);
        }
      }
      __syncwarp();
    } else if (warp == 10) {
      // ---------------------------------------------------------------- PV issuer
      constexpr uint32_t idO = ptx::idesc_bf16(kPtRows, D, false, true);
      // only the first and last tile can hold V rows that may be anything; the warp zeroes them
      // (their weights are zero too) before its lane 0 issues that tile.  A loop that kept all
      // lanes together for every tile cost 3 %
      auto edge = [&](int t) -> bool {
        const int j0 = (t_begin + t) * kPtKeys;
        return t >= 0 && t < nt && (j0 < lo || j0 + kPtKeys > key_end);
      };
      auto zero_rows = [&](int t) {
        const int vs = (kt + t) % kPtSlots, j0 = (t_begin + t) * kPtKeys;
        if (!ptx::mbar_wait(&bars->v_full[vs], ((kt + t) / kPtSlots) & 1, abort_flag)) return;
        for (int r = lane; r < kPtKeys; r += 32)
          if (j0 + r < lo || j0 + r >= key_end)
            for (int db = 0; db < C::kDB; ++db) {
              uint4* row =
                  reinterpret_cast<uint4*>(sV + vs * C::kTileBytes + (r >> 3) * C::kGroup + db * 1024 + (r & 7) * 128);
#pragma unroll
              for (int k = 0; k < 8; ++k) row[k] = make_uint4(0, 0, 0, 0);
            }
        ptx::fence_proxy_async_smem();
      };
      auto issue = [&](int t) -> bool {
        const int vs = (kt + t) % kPtSlots;
        if (!ptx::mbar_wait(&bars->v_full[vs], ((kt + t) / kPtSlots) & 1, abort_flag)) return false;
        const uint64_t vd = ptx::sdesc_sw128(ptx::smem_addr(sV + vs * C::kTileBytes), 1024, C::kGroup);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (t >= ntx[x]) continue;
          const unsigned tx = done_x[x] + t;
          const int buf = tx & 1;
          if (!ptx::mbar_wait(&bars->p_full[x][buf], (tx >> 1) & 1, abort_flag)) return false;
          ptx::tc_fence_after();
          pt_pv_product(tmem + C::kColO + x * kPtRows, tmem + x * kPtRows + buf * kPtKeys, vd, 2 * C::kGroup / 16, idO,
                        t > 0 ? 1u : 0u);  // P: 8 columns per 16 keys
          ptx::mma_commit(&bars->pv_done[x][buf]);
        }
        ptx::mma_commit(&bars->v_empty[vs]);
        return true;
      };
      const int last = nt - 1;
      // one copy of the loop's code: a kernel of few steps pays for each line that it fetches first
#pragma unroll 1
      for (int part = 0, t = 0; part < 2; ++part) {
        const int from = part == 0 ? 0 : last, to = part == 0 ? last : nt;
        if (from < to && edge(from)) zero_rows(from);
        __syncwarp();
        // the piece before's O has been read
        if (kStream && part == 0 && pieces > 0 && nt > 0)
          for (int x = 0; x < 2; ++x)
            ok = __all_sync(0xffffffffu, ok && ptx::mbar_wait(&bars->o_free[x], (pieces - 1) & 1, abort_flag));
        if (lane == 0)
          for (; ok && t < to; ++t) ok = issue(t);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      if (lane == 0 && nt > 0) {
        ptx::mma_commit(&bars->o_done);
        pt_drain(&bars->o_done, pieces & 1, abort_flag);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- softmax rows
      const int x = (warp - 2) >> 2;
      const int q4 = warp & 3;
      const int r = q4 * 32 + lane;
      const int g = r / NT, node = pt_of(i0, x) + r % NT;
      const bool valid = x < pa.tiles && r < rows_used && node < n_act;
      const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
      const uint32_t colS = tmem + lane_base + x * kPtRows;
      const uint32_t colO = tmem + lane_base + C::kColO + x * kPtRows;
      const int ntm = pt_of(ntx, x);
      const unsigned dx = pt_of(done_x, x);
      // the row sees [wlo, whi) and, in a tree, its ancestors; rows that are no row see everything
      // (their results go nowhere)
      int wlo = 0, whi = 0x7fffffff;
      if (valid) {
        int depth = node;
        if (a.parent) {
          whi = P;
          if (a.window > 0) {
            depth = 0;
            for (int at = s_par[node]; at >= 0; at = s_par[at]) ++depth;  // parents fall: it ends
          }
        } else {
          whi = P + node + 1;
        }
        if (a.window > 0) wlo = max(0, P + depth - a.window + 1);  // at least 0: wlo - j0 fits an int
      }
      const float c = kCap == kLargeCap ? kLog2e : kCap ? a.cap * kLog2e : a.scale * kLog2e;
      const float ck = kCap == kLargeCap ? 1.f / a.cap : kCap ? 2.f * kLog2e * a.scale / a.cap : 0.f;
      for (int t = 0; ok && t < ntm; ++t) {
        const unsigned tx = dx + t;
        const int buf = tx & 1;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars->s_full[x][buf], (tx >> 1) & 1, abort_flag));
        if (!ok) break;
        ptx::tc_fence_after();
        const int j0 = (t_begin + t) * kPtKeys;
        uint64_t vis = ~0ull;
        if (j0 < wlo || j0 + kPtKeys > whi) {
          vis = pt_bits(wlo - j0, whi - j0);
          if (a.parent) {
            int steps = a.window > 0 ? a.window : kMaxNodes + 1;
            for (int at = node; at >= 0 && steps > 0; at = s_par[at], --steps) {
              const int j = P + at - j0;
              if (j < 0) break;  // ancestors only go down from here
              if (j < kPtKeys) vis |= 1ull << j;
            }
          }
        }
        float sv[64];
        ptx::tmem_ld32(colS + buf * kPtKeys, sv);
        ptx::tmem_ld32(colS + buf * kPtKeys + 32, sv + 32);
        ptx::tmem_wait_ld();
        if constexpr (kCap == kTanhCap) {
          if (vis != ~0ull) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (!((vis >> j) & 1ull)) sv[j] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < 64; j += 4) soft_tanh4(sv + j, ck);
        } else if constexpr (kCap == kLargeCap) {
          // nearly all scores lie below 0.45 of such a cap; where one does not, the tile is read again
          float z_max = 0.f;
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            const float t = sv[j] * a.scale, x = t * ck, z = x * x;
            z_max = fmaxf(z_max, z);
            sv[j] = fmaf(t * z, tanh_tail(z), t);
          }
          if (__any_sync(0xffffffffu, z_max >= kTanhNear)) {
            ptx::tmem_ld32(colS + buf * kPtKeys, sv);
            ptx::tmem_ld32(colS + buf * kPtKeys + 32, sv + 32);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 64; ++j) sv[j] = capped_score(sv[j] * a.scale, a.cap, ck);
          }
        }
        if (vis != ~0ull) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (!((vis >> j) & 1ull)) sv[j] = -INFINITY;
        }
        // P = 2^(c S - m_run) against a running reference that moves (with a rescale of O) only
        // when a score exceeds it by 2^8: such a score brings the tile's sum to 2^8, so the
        // maximum is taken only then and for the first tile with a visible key
        float alpha = 1.f;
        bool need = false, checked = false;
        if (m_run == -INFINITY) {
          m_run = pt_max64(sv) * c;
          checked = true;
        }
        uint32_t pw[32];
        float lsum;
        for (;;) {
          lsum = pt_exp64(sv, c, m_run, pw);
          if (checked || lsum < kPtRescaleSum) break;
          checked = true;
          const float tms = pt_max64(sv) * c;
          if (!(tms > m_run + kPtRescaleLog2)) break;
          alpha = ptx::ex2(m_run - tms);
          need = true;
          m_run = tms;
        }
        ptx::tmem_st32u(colS + buf * kPtKeys, pw);
        if (__any_sync(0xffffffffu, need) && t > 0) {
          // O_X must hold all of PV_X(t - 1) before it is rescaled
          ok = __all_sync(0xffffffffu,
                          ptx::mbar_wait(&bars->pv_done[x][(tx - 1) & 1], ((tx - 1) >> 1) & 1, abort_flag));
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            float ov[32];
            ptx::tmem_ld32(colO + c0, ov);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) ov[k] *= alpha;
            ptx::tmem_st32(colO + c0, ov);
          }
        }
        l_run = l_run * alpha + lsum;
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->p_full[x][buf]);
      }
      // ---- epilogue: every MMA is complete at o_done
      if (isnan(l_run)) m_run = l_run;  // a NaN query's part: no part without a visible key, which merges leave out
      if (nt > 0) {
        ok = ok && __all_sync(0xffffffffu, ptx::mbar_wait(&bars->o_done, pieces & 1, abort_flag));
        have_o = ok && ntm > 0;
        if (ok) ptx::tc_fence_after();
      }
      // read here, not kept through the loop
      const volatile PtPiece& at = s_piece[np % kPtPieces];
      const bool whole = kStream && at.c1 <= at.c0;
      const int R = x * kPtRows + r;
      const size_t slot = kStream ? (size_t)at.slot : cta;
      const float inv = whole && l_run > 0.f ? 1.f / l_run : 0.f;
      const size_t orow = (((size_t)b * a.Hq + hk * a.G + g) * a.N + node) * a.D;
      float4* part = whole ? nullptr : reinterpret_cast<float4*>(a.ws_o) + slot * (D / 4) * 2 * kPtRows + R;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        if (x >= pa.tiles) break;
        float ov[32];
        if (have_o) {
          ptx::tmem_ld32(colO + c0, ov);
          ptx::tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) ov[k] = 0.f;
        }
        if (whole) {
          if (valid && c0 < a.D) {
            uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + orow + c0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[k] = make_uint4(ptx::cvt_bf16x2(ov[8 * k + 0] * inv, ov[8 * k + 1] * inv),
                                  ptx::cvt_bf16x2(ov[8 * k + 2] * inv, ov[8 * k + 3] * inv),
                                  ptx::cvt_bf16x2(ov[8 * k + 4] * inv, ov[8 * k + 5] * inv),
                                  ptx::cvt_bf16x2(ov[8 * k + 6] * inv, ov[8 * k + 7] * inv));
          }
        } else {
          // partial O as [D / 4][256 rows] of four columns: a warp stores 512 bytes in a row
#pragma unroll
          for (int k = 0; k < 8; ++k)
            __stcg(part + (size_t)(c0 / 4 + k) * 2 * kPtRows,
                   make_float4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]));
        }
      }
      if (!whole)
        __stcg(a.ws_ml + slot * 2 * kPtRows + R, make_float2(have_o ? m_run : -INFINITY, have_o ? l_run : 0.f));
      ptx::tc_fence_before();
      __syncwarp();
      if (kStream && nt > 0 && lane == 0) ptx::mbar_arrive(&bars->o_free[x]);
    }
    __syncwarp();

    if constexpr (kStream) {
      // only the softmax warps take part; the others go on to the next piece
      const volatile PtPiece& at = s_piece[np % kPtPieces];
      const int c0 = at.c0, c1 = at.c1;
      if (c0 < c1 && warp >= 2 && warp < 10) {
        __threadfence();
        softmax_sync();
        if (threadIdx.x == 64) {
          s_last = ptx::atom_add_acq_rel_gpu(&a.cnt[c0], 1u) == (unsigned)(c1 - c0);
          if (s_last) a.cnt[c0] = 0u;
          __threadfence();
        }
        softmax_sync();
        if (s_last) {
          const int x = (warp - 2) >> 2, r = (warp & 3) * 32 + lane, R = x * kPtRows + r;
          const int g = r / NT, node = pt_of(i0, x) + r % NT;
          if (r < rows_used && node < n_act) {
            auto place = [&](int cc) -> size_t { return cc == c0 ? at.slot0 : 2 * cc; };
            auto stats = [&](int cc) -> float2 { return __ldcg(&a.ws_ml[place(cc) * 2 * kPtRows + R]); };
            float M = -INFINITY, L = 0.f;
#pragma unroll 4
            for (int cc = c0; cc <= c1; ++cc) M = fmaxf(M, stats(cc).x);
#pragma unroll 4
            for (int cc = c0; cc <= c1; ++cc) {
              const float2 ml = stats(cc);
              if (ml.x != -INFINITY) L = fmaf(ptx::ex2(ml.x - M), ml.y, L);
            }
            const float inv = L > 0.f ? 1.f / L : 0.f;
            const size_t orow = (((size_t)b * a.Hq + hk * a.G + g) * a.N + node) * a.D;
#pragma unroll 1
            for (int col = 0; col < a.D; col += 32) {
              float ov[32];
#pragma unroll
              for (int k = 0; k < 32; ++k) ov[k] = 0.f;
              // two parts' loads in flight together
              for (int cc = c0; cc <= c1; cc += 2) {
                float wt[2];
                float4 v[2][8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const int from = min(cc + u, c1);
                  const float2 ml = stats(from);
                  wt[u] = cc + u > c1 || ml.x == -INFINITY ? 0.f : ptx::ex2(ml.x - M);
                  const float4* src = reinterpret_cast<const float4*>(a.ws_o) +
                                      (place(from) * (D / 4) + col / 4) * 2 * kPtRows + R;
#pragma unroll
                  for (int k = 0; k < 8; ++k) v[u][k] = __ldcg(src + (size_t)k * 2 * kPtRows);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                  for (int k = 0; k < 8; ++k) {
                    ov[4 * k] = fmaf(wt[u], v[u][k].x, ov[4 * k]);
                    ov[4 * k + 1] = fmaf(wt[u], v[u][k].y, ov[4 * k + 1]);
                    ov[4 * k + 2] = fmaf(wt[u], v[u][k].z, ov[4 * k + 2]);
                    ov[4 * k + 3] = fmaf(wt[u], v[u][k].w, ov[4 * k + 3]);
                  }
              }
              uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + orow + col);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                dst[k] = make_uint4(ptx::cvt_bf16x2(ov[8 * k + 0] * inv, ov[8 * k + 1] * inv),
                                    ptx::cvt_bf16x2(ov[8 * k + 2] * inv, ov[8 * k + 3] * inv),
                                    ptx::cvt_bf16x2(ov[8 * k + 4] * inv, ov[8 * k + 5] * inv),
                                    ptx::cvt_bf16x2(ov[8 * k + 6] * inv, ov[8 * k + 7] * inv));
            }
          }
        }
      }
    } else {
      // the parts form one cluster, and each CTA merges its share of the rows.  They meet in L2, not in
      // distributed shared memory: 64 KB a CTA through a cluster took 2.8 us, stored or read
      ptx::cluster_sync();
      const int S = pa.splits;
      const int share = (pa.tiles * kPtRows + S - 1) / S;
      const int r0 = split * share, rows = min(pa.tiles * kPtRows, r0 + share) - r0;
      const size_t first = cta - split;
      for (int item = threadIdx.x; item < rows * (a.D / 4); item += kPtThreads) {
        const int ch = item / rows, R = r0 + item - ch * rows;
        const int x = R >= kPtRows ? 1 : 0, r = R - x * kPtRows;
        const int g = r / NT, node = pt_of(i0, x) + r % NT;
        if (r >= rows_used || node >= n_act) continue;
        float2 mlv[kPtMaxSplits];
        float4 xv[kPtMaxSplits];
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int s2 = 0; s2 < kPtMaxSplits; ++s2)
          if (s2 < S) {
            mlv[s2] = __ldcg(a.ws_ml + (first + s2) * 2 * kPtRows + R);
            xv[s2] = __ldcg(reinterpret_cast<const float4*>(a.ws_o) + ((first + s2) * (D / 4) + ch) * 2 * kPtRows + R);
          }
#pragma unroll
        for (int s2 = 0; s2 < kPtMaxSplits; ++s2)
          if (s2 < S) M = fmaxf(M, mlv[s2].x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s2 = 0; s2 < kPtMaxSplits; ++s2)
          if (s2 < S && mlv[s2].x != -INFINITY) {
            const float w = ptx::ex2(mlv[s2].x - M);
            L = fmaf(mlv[s2].y, w, L);
            acc.x = fmaf(w, xv[s2].x, acc.x);
            acc.y = fmaf(w, xv[s2].y, acc.y);
            acc.z = fmaf(w, xv[s2].z, acc.z);
            acc.w = fmaf(w, xv[s2].w, acc.w);
          }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const size_t o = (((size_t)b * a.Hq + hk * a.G + g) * a.N + node) * a.D + ch * 4;
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + o) =
            make_uint2(ptx::cvt_bf16x2(acc.x * inv, acc.y * inv), ptx::cvt_bf16x2(acc.z * inv, acc.w * inv));
      }
    }
    if constexpr (kStream) {
      __syncwarp();
      if (warp != 0 && lane == 0) ptx::mbar_arrive(&bars->piece_empty[np % kPtPieces]);
    }
    kt += nt;
    done_x[0] += ntx[0];
    done_x[1] += ntx[1];
    pieces += nt > 0;
    if (!kStream) break;
  }
  if (kStream && threadIdx.x == 0) drain();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && bars->abort) set_dev_status(a.dev_status, TV_DEV_TIMEOUT);
}

// ---- host side

typedef CUresult (*PtEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static bool pt_encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                      const cuuint32_t* box) {
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
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

struct PtPlan {
  int NT, tiles, MP, splits, grid;  // splits 0: persistent grid
  size_t slots, bytes;        // workspace: partial results
};

// Clusters of s CTAs that can be resident at once on the current device (known per device and s).
static int pt_clusters(int D, int s) {
  static std::atomic<int> known[64][kPtMaxSplits + 1];  // count + 1; 0 = not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return paged_device_sms() / s;
  int n = known[dev][s].load(std::memory_order_relaxed) - 1;
  if (n < 0) {
    // every instance takes one CTA per SM, so one stands for all
    const void* fn = reinterpret_cast<const void*>(paged_tc_kernel<128, kNoCap, false>);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s * 64, 1, 1);
    cfg.blockDim = dim3(kPtThreads, 1, 1);
    cfg.dynamicSmemBytes = PtCfg<128>::kSmemAlloc;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)s;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, PtCfg<128>::kSmemAlloc) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess)
      n = paged_device_sms() / s;
    known[dev][s].store(n + 1, std::memory_order_relaxed);
  }
  return n;
}

static PtPlan pt_plan(int B, int Hq, int Hkv, int D, int N, int share) {
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
  const size_t n = pt_plan(B, Hq, Hkv, D, N, paged_device_sms()).bytes;
  return {n, n};
}

template <int D, int kCap, bool kStream>
static cudaError_t launch_pt(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a,
                             const PtPlan& p, cudaStream_t stream) {
  constexpr int smem = PtCfg<D>::kSmemAlloc;
  cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<D, kCap, kStream>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem);
  if (e != cudaSuccess) return e;
  const PtArgs pa{p.NT, p.tiles, p.MP, p.splits, a.D == 128};
  if (kStream)
    return launch_pdl(paged_tc_kernel<D, kCap, kStream>, dim3((unsigned)p.grid), dim3(kPtThreads), smem, stream,
                      nullptr, 0, mq, mk, mv, a, pa);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  return launch_pdl(paged_tc_kernel<D, kCap, kStream>, dim3((unsigned)(p.MP * p.splits), (unsigned)a.Hkv, (unsigned)a.B),
                    dim3(kPtThreads), smem, stream, attr, 1, mq, mk, mv, a, pa);
}

template <int D, int kCap>
static cudaError_t launch_pt_c(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a,
                               const PtPlan& p, cudaStream_t stream) {
  return p.splits ? launch_pt<D, kCap, false>(mq, mk, mv, a, p, stream)
                  : launch_pt<D, kCap, true>(mq, mk, mv, a, p, stream);
}
template <int D>
static cudaError_t launch_pt_d(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a,
                               const PtPlan& p, cudaStream_t stream) {
  switch (cap_mode(a.cap)) {
    case kLargeCap:
      return launch_pt_c<D, kLargeCap>(mq, mk, mv, a, p, stream);
    case kTanhCap:
      return launch_pt_c<D, kTanhCap>(mq, mk, mv, a, p, stream);
    default:
      return launch_pt_c<D, kNoCap>(mq, mk, mv, a, p, stream);
  }
}

cudaError_t launch_paged_tc(PagedAttn a, char* ws, cudaStream_t stream) {
  const PtPlan p = pt_plan(a.B, a.Hq, a.Hkv, a.D, a.N, a.sms);
  a.cnt = reinterpret_cast<unsigned*>(ws);
  a.ws_ml = reinterpret_cast<float2*>(ws + kPagedCntBytes);
  a.ws_o = reinterpret_cast<float*>(ws + kPagedCntBytes + p.slots * 2 * kPtRows * 8);
  CUtensorMap mq, mk, mv;
  if (!pt_tmap(&mq, a.q, a.D, a.N, (long long)a.B * a.Hq, p.NT) || !paged_kv_tmap(&mk, a.k, a) ||
      !paged_kv_tmap(&mv, a.v, a))
    return cudaErrorInvalidValue;
  return a.D <= 64 ? launch_pt_d<64>(mq, mk, mv, a, p, stream) : launch_pt_d<128>(mq, mk, mv, a, p, stream);
}

}  // namespace tv
