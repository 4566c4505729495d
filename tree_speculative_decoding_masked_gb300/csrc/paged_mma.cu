// Attention of few rows over a paged KV cache (single tokens, short chunks, small trees), bf16.
//
// With at most 32 query rows a KV head every key is read for a handful of products: the
// work is a stream of K and V pages from HBM and the kernel's job is to keep enough of
// them in flight.  One warp per CTA fetches 64-key tiles by TMA (a box per page piece) into
// a ring and runs ahead across sequences and heads; four warps (times kMT row groups of 16)
// take 16 keys of a tile each:
//   S = Q K^T (16 rows x 16 keys) and O += P V by warp-level MMAs on shared memory,
// whose rate is an order of magnitude above what the stream needs, while a tcgen05 product
// would spend a 128-row tile on 4 rows.  Each warp keeps its own running reference and sums
// (32 bits) and its own O in registers; P is rounded to bf16 for the second product.  The
// four O's are added in warp order when the unit ends, so results do not depend on timing.
//
// The keys of all (sequence, KV head) units are divided equally over a persistent grid
// (paged.cuh); parts of cut units are merged through the workspace.
#include "paged.cuh"

namespace tv {

constexpr int kPmKeys = 64;
constexpr int kPmMerge = 8;   // parts whose loads are in flight together
constexpr int kPmMinTiles = 2;  // tiles of a CTA's range: fewer only add parts to merge

template <int kD, int kMT>
struct PmCfg {
  static constexpr int kDB = kD / 64;
  static constexpr int kRT = 16 * kMT;
  static constexpr int kConsumers = 128 * kMT;
  static constexpr int kThreads = kConsumers + 32;
  static constexpr int kBlock = kPmKeys * 128;          // one 64-column block of a K or V tile
  static constexpr int kStage = 2 * kDB * kBlock;       // K then V
  static constexpr int kCtas = kD <= 128 && kMT == 1 ? 2 : 1;  // per SM
  static constexpr int kStages = kD == 64 ? (kMT == 1 ? 6 : 8) : kD == 128 ? (kMT == 1 ? 3 : 5) : (kMT == 1 ? 3 : 2);
  static constexpr int kQStride = kD * 2 + 16;          // bytes: ldmatrix rows on different banks
  // the unit's queries, masks and tree; its O at the end
  static constexpr int kOffU = kStages * kStage;
  static constexpr int kOffVis = kOffU + kRT * kQStride;
  static constexpr int kOffPar = kOffVis + kRT * (kMaxNodes / 32) * 4;
  static constexpr int kInBytes = kOffPar + kMaxNodes * 4 - kOffU;
  static constexpr int kOBytes = kRT * kD * 4;
  static constexpr int kOffBar = kOffU + (kInBytes > kOBytes ? kInBytes : kOBytes);
  static constexpr int kSmem = kOffBar + 256 + 1024;
  static_assert(kCtas * (kSmem + 2048) <= 233472, "shared memory per SM");
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
__device__ __forceinline__ void pm_ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void pm_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The next unit with work in this CTA's range [pos, end): its sequence, KV head, row tile and
// tiles [t0, t1).  The producer and the consumers walk the same sequence of them.
struct PmWalk {
  long long pos, end, base, u0, u1;
  int b, hk, rt, P, n, n_act, loaded, t0, t1;
};

template <int kRT>
__device__ __forceinline__ bool pm_next(const PagedAttn& a, PmWalk& w) {
  while (w.pos < w.end && w.b < a.B) {
    if (w.loaded != w.b) {
      bool bad;
      w.P = a.prefix_len[w.b];
      w.n = paged_rows(a, w.b, w.P, &bad);
      w.loaded = w.b;
      w.n_act = -1;
    }
    const int T_u = unit_tiles(a, w.P, w.n, w.rt, kRT, kPmKeys);
    w.u0 = w.base;
    w.base += T_u;
    if (w.pos < w.base) {
      w.u1 = w.base;
      w.t0 = (int)(w.pos - w.u0);
      w.t1 = (int)(min(w.base, w.end) - w.u0);
      w.pos = w.u0 + w.t1;
      return true;
    }
    if (++w.rt * kRT >= w.n * a.G) {
      w.rt = 0;
      if (++w.hk >= a.Hkv) w.hk = 0, ++w.b;
    }
  }
  return false;
}
// step over the unit that pm_next returned
template <int kRT>
__device__ __forceinline__ void pm_step(const PagedAttn& a, PmWalk& w) {
  if (++w.rt * kRT >= w.n * a.G) {
    w.rt = 0;
    if (++w.hk >= a.Hkv) w.hk = 0, ++w.b;
  }
}

template <int kD, int kMT, bool kCap>
__global__ void __launch_bounds__(PmCfg<kD, kMT>::kThreads, PmCfg<kD, kMT>::kCtas)
    paged_mma_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, PagedAttn a) {
  using C = PmCfg<kD, kMT>;
  ptx::griddep_launch_dependents();
  extern __shared__ unsigned char pm_raw[];
  unsigned char* sm = pm_raw + ((1024u - (ptx::smem_addr(pm_raw) & 1023u)) & 1023u);
  PmBars* bars = reinterpret_cast<PmBars*>(sm + C::kOffBar);
  volatile int* abort_flag = &bars->abort;
  __shared__ unsigned long long s_red[34];
  __shared__ int s_lo[C::kRT], s_hi[C::kRT], s_first_pad, s_last;
  __shared__ float s_m[4][C::kRT], s_l[4][C::kRT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&bars->full[s], 1);
      ptx::mbar_init(&bars->empty[s], 4 * kMT);
    }
    bars->abort = 0;
    ptx::fence_mbar_init();
  }
  ptx::griddep_wait();
  __syncthreads();
  const PagedSpan sp = paged_span(a, C::kRT, kPmKeys, kPmMinTiles, s_red);
  __syncthreads();
  PmWalk w{};
  w.pos = sp.per * blockIdx.x;
  w.end = min(sp.W, w.pos + sp.per);
  w.base = sp.base;
  w.b = sp.b;
  w.loaded = -1;
  int it = 0;  // tiles so far: ring slot it % kStages

  if (warp == 4 * kMT) {
    // ------------------------------------------------------------------ producer
    // lane: K or V, column block db, page piece pi of the tile (D = 256: two rounds of pieces)
    const int box_shift = min(a.page_shift, 6), pieces = kPmKeys >> box_shift;
    const int box_rows = 1 << box_shift;
    const uint32_t box_bytes = 128u << box_shift;
    const int page_mask = (1 << a.page_shift) - 1;
    int issued = 0;
    while (pm_next<C::kRT>(a, w)) {
      if (w.n_act < 0) {
        int pad = w.n;
        if (a.parent)
          for (int t = lane; t < w.n; t += 32)
            if (t > 0 && t < pad && a.parent[(size_t)w.b * a.N + t] == -1) pad = t;
        w.n_act = __reduce_min_sync(0xffffffffu, pad);
      }
      const int rows = unit_rows(a, w.n, w.rt, C::kRT);
      const int lo = unit_lo(a, w.P, w.rt, C::kRT), tile0 = lo / kPmKeys;
      const int hi = min(w.P + w.n_act, w.P + (w.rt * C::kRT + rows - 1) / a.G + 1);
      const int32_t* table = a.table + (size_t)w.b * a.max_pages;
      // the page of piece `lane` (lanes 0..pieces-1) of tile t, -1 where no row is needed or the page is bad
      auto lookup = [&](int t) -> int {
        const int j = (tile0 + t) * kPmKeys + (lane << box_shift);
        if (t >= w.t1 || lane >= pieces || j >= hi || j + box_rows <= lo) return -1;
        const int page = table[j >> a.page_shift];
        if (page < 0 || page >= a.num_pages) {
          set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
          return -1;
        }
        return page;
      };
      int next = lookup(w.t0);
      for (int t = w.t0; t < w.t1; ++t, ++it) {
        const int page = next;  // read one tile ahead
        next = lookup(t + 1);
        const int slot = it % C::kStages;
        bool ok = true;
        if (it >= C::kStages) ok = ptx::mbar_wait(&bars->empty[slot], ((it / C::kStages) - 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) continue;  // aborted: no more copies; the consumers do not wait either
        issued = it + 1;
        const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) ptx::mbar_arrive_expect_tx(&bars->full[slot], __popc(have) * box_bytes * 2 * C::kDB);
        __syncwarp();
        unsigned char* stage = sm + slot * C::kStage;
        // box e: column block and K / V of one piece, its page from the piece's lane
        for (int e0 = 0; e0 < pieces * 2 * C::kDB; e0 += 32) {
          const int e = e0 + lane, pi = e / (2 * C::kDB), part = e % (2 * C::kDB);
          const int pg = __shfl_sync(0xffffffffu, page, pi & 31);
          if (e < pieces * 2 * C::kDB && pg >= 0) {
            const int db = part >> 1, j = (tile0 + t) * kPmKeys + (pi << box_shift);
            unsigned char* dst = stage + ((part & 1) * C::kDB + db) * C::kBlock + (pi << box_shift) * 128;
            ptx::tma_load_3d(dst, (part & 1) ? &tmV : &tmK, &bars->full[slot], db * 64, j & page_mask,
                             pg * a.Hkv + w.hk);
          }
        }
        __syncwarp();
      }
      pm_step<C::kRT>(a, w);
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
    const int wk = warp & 3, mt = warp >> 2;  // key quarter, row group
    const int ct = threadIdx.x;
    unsigned char* sQ = sm + C::kOffU;
    uint32_t(*s_vis)[kMaxNodes / 32] = reinterpret_cast<uint32_t(*)[kMaxNodes / 32]>(sm + C::kOffVis);
    int* s_par = reinterpret_cast<int*>(sm + C::kOffPar);
    float* sO = reinterpret_cast<float*>(sm + C::kOffU);
    const int rg = lane >> 2, cg = (lane & 3) * 2;  // this lane's rows rg, rg + 8 and key / column pairs
    const float c = kCap ? a.cap * kLog2e : a.scale * kLog2e;
    const float ck = kCap ? 2.f * kLog2e * a.scale / a.cap : 0.f;
    bool ok = true;
    while (pm_next<C::kRT>(a, w)) {
      const int rows = unit_rows(a, w.n, w.rt, C::kRT), r0 = w.rt * C::kRT;
      const int lo = unit_lo(a, w.P, w.rt, C::kRT), tile0 = lo / kPmKeys;
      cons_sync();  // the previous unit's O has been read
      int n_act = w.n;
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
      for (int e = ct; e < C::kRT * (kD / 8); e += C::kConsumers) {
        const int rr = e / (kD / 8), ch = e % (kD / 8), i = (r0 + rr) / a.G, g = (r0 + rr) % a.G;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (rr < rows && i < n_act && ch * 8 < a.D)
          v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                              (((size_t)w.b * a.Hq + w.hk * a.G + g) * a.N + i) * a.D + ch * 8);
        *reinterpret_cast<uint4*>(sQ + rr * C::kQStride + ch * 16) = v;
      }
      if (ct < C::kRT) {
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
      // every row of this warp's group sees all of [full_lo, full_hi)
      const int full_lo = __reduce_max_sync(0xffffffffu, lane < 16 ? s_lo[mt * 16 + lane] : 0);
      const int full_hi = __reduce_min_sync(0xffffffffu, lane < 16 ? s_hi[mt * 16 + lane] : 0x7fffffff);
      const uint32_t qaddr = ptx::smem_addr(sQ + (mt * 16 + (lane & 15)) * C::kQStride + (lane >> 4) * 16);
      uint32_t qf[kD <= 128 ? kD / 16 : 1][4];
      if constexpr (kD <= 128) {
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) pm_ldsm4(qf[kk], qaddr + kk * 32);
      }
      float o[kD / 8][4];
#pragma unroll
      for (int k = 0; k < kD / 8; ++k)
#pragma unroll
        for (int u = 0; u < 4; ++u) o[k][u] = 0.f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

      for (int t = w.t0; t < w.t1; ++t, ++it) {
        const int slot = it % C::kStages;
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars->full[slot], (it / C::kStages) & 1, abort_flag));
        if (!ok) continue;
        const int j0 = (tile0 + t) * kPmKeys + wk * 16;  // this warp's 16 keys
        unsigned char* sK = sm + slot * C::kStage;
        unsigned char* sV = sK + C::kDB * C::kBlock;
        if (j0 >= hi || j0 + 16 <= lo) {  // none of them
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bars->empty[slot]);
          continue;
        }
        const int krow = wk * 16 + (lane & 7) + ((lane >> 4) & 1) * 8;
        const uint32_t kaddr = ptx::smem_addr(sK + krow * 128);
        float s[2][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) s[0][u] = s[1][u] = 0.f;
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          uint32_t kf[4];
          const int ch = (kk & 3) * 2 + ((lane >> 3) & 1);
          pm_ldsm4(kf, kaddr + (kk >> 2) * C::kBlock + ((ch ^ (krow & 7)) << 4));
          if constexpr (kD <= 128) {
            pm_mma(s[0], qf[kk], kf[0], kf[1]);
            pm_mma(s[1], qf[kk], kf[2], kf[3]);
          } else {
            uint32_t qk[4];
            pm_ldsm4(qk, qaddr + kk * 32);
            pm_mma(s[0], qk, kf[0], kf[1]);
            pm_mma(s[1], qk, kf[2], kf[3]);
          }
        }
        if constexpr (kCap) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int u = 0; u < 4; ++u) s[h][u] = soft_tanh(s[h][u] * ck);
        }
        const bool edge = j0 < lo || j0 + 16 > hi;
        if (j0 < full_lo || j0 + 16 > full_hi || edge) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int rr = mt * 16 + rg + (u >> 1) * 8, j = j0 + h * 8 + cg + (u & 1);
              bool vis = j >= s_lo[rr] && j < s_hi[rr];
              if (!vis && a.parent && j >= w.P && j < hi)
                vis = (s_vis[rr][(j - w.P) >> 5] >> ((j - w.P) & 31)) & 1u;
              if (!vis) s[h][u] = -INFINITY;
            }
          if (edge) {
            // V rows that were not fetched or may hold anything, NaN included: zero
            for (int e = lane; e < 16 * C::kDB * 8; e += 32) {
              const int rr = e / (C::kDB * 8), rest = e % (C::kDB * 8);
              if (j0 + rr < lo || j0 + rr >= hi)
                *reinterpret_cast<uint4*>(sV + (rest >> 3) * C::kBlock + (wk * 16 + rr) * 128 + (rest & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async_smem();  // before the slot is refilled
            __syncwarp();
          }
        }
        // the running reference moves when a score exceeds it by 2^8
        uint32_t pf[4];
        bool grow = false;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            s[h][u] *= c;
            grow |= s[h][u] > m[u >> 1] + 8.f;
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float mx = fmaxf(fmaxf(s[0][2 * q], s[0][2 * q + 1]), fmaxf(s[1][2 * q], s[1][2 * q + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            if (mx > m[q]) {
              const float f = ptx::ex2(m[q] - mx);  // 0 from -inf
              m[q] = mx;
              l[q] *= f;
#pragma unroll
              for (int k = 0; k < kD / 8; ++k) {
                o[k][2 * q] *= f;
                o[k][2 * q + 1] *= f;
              }
            }
          }
        }
        const float b0 = m[0] == -INFINITY ? 0.f : m[0], b1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float e0 = ptx::ex2(s[h][0] - b0), e1 = ptx::ex2(s[h][1] - b0);
          const float e2 = ptx::ex2(s[h][2] - b1), e3 = ptx::ex2(s[h][3] - b1);
          l[0] += e0 + e1;
          l[1] += e2 + e3;
          pf[2 * h] = ptx::cvt_bf16x2(e0, e1);
          pf[2 * h + 1] = ptx::cvt_bf16x2(e2, e3);
        }
        const int vrow = wk * 16 + (lane & 15);
        const uint32_t vaddr = ptx::smem_addr(sV + vrow * 128);
#pragma unroll
        for (int nn = 0; nn < kD / 16; ++nn) {
          uint32_t vf[4];
          const int ch = (nn & 3) * 2 + (lane >> 4);
          pm_ldsm4t(vf, vaddr + (nn >> 2) * C::kBlock + ((ch ^ (vrow & 7)) << 4));
          pm_mma(o[2 * nn], pf, vf[0], vf[1]);
          pm_mma(o[2 * nn + 1], pf, vf[2], vf[3]);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->empty[slot]);
      }

      // ---- the four key quarters' results, added in order
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        l[q] += __shfl_xor_sync(0xffffffffu, l[q], 1);
        l[q] += __shfl_xor_sync(0xffffffffu, l[q], 2);
        if ((lane & 3) == 0) {
          s_m[wk][mt * 16 + rg + 8 * q] = m[q];
          s_l[wk][mt * 16 + rg + 8 * q] = l[q];
        }
      }
      cons_sync();  // and every warp is done with the queries and masks, which O now overwrites
      float f[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int rr = mt * 16 + rg + 8 * q;
        const float M = fmaxf(fmaxf(s_m[0][rr], s_m[1][rr]), fmaxf(s_m[2][rr], s_m[3][rr]));
        f[q] = m[q] == -INFINITY ? 0.f : ptx::ex2(m[q] - M);
      }
      for (int k = 0; k < 4; ++k) {
        if (wk == k) {
#pragma unroll
          for (int d = 0; d < kD / 8; ++d)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float2* at = reinterpret_cast<float2*>(sO + (mt * 16 + rg + 8 * q) * kD + d * 8 + cg);
              const float2 was = k ? *at : make_float2(0.f, 0.f);
              *at = make_float2(fmaf(f[q], o[d][2 * q], was.x), fmaf(f[q], o[d][2 * q + 1], was.y));
            }
        }
        cons_sync();
      }
      // ---- write the unit, or this CTA's part of it
      const long long c0 = w.u0 / sp.per, c1 = (w.u1 - 1) / sp.per;
      const int slot = unit_slot(blockIdx.x, sp.per, w.u0);
      const int quads = a.D / 4;
      for (int e = ct; e < rows * quads; e += C::kConsumers) {
        const int rr = e / quads, ch = e % quads, i = (r0 + rr) / a.G, g = (r0 + rr) % a.G;
        if (i >= n_act) continue;
        const float4 v = *reinterpret_cast<const float4*>(sO + rr * kD + ch * 4);
        const float M = fmaxf(fmaxf(s_m[0][rr], s_m[1][rr]), fmaxf(s_m[2][rr], s_m[3][rr]));
        float L = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (s_m[k][rr] != -INFINITY) L = fmaf(s_l[k][rr], ptx::ex2(s_m[k][rr] - M), L);
        if (c0 == c1) {
          const float inv = 1.f / L;
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) +
                                    (((size_t)w.b * a.Hq + w.hk * a.G + g) * a.N + i) * a.D + ch * 4) =
              make_uint2(ptx::cvt_bf16x2(v.x * inv, v.y * inv), ptx::cvt_bf16x2(v.z * inv, v.w * inv));
        } else {
          __stcg(reinterpret_cast<float4*>(a.ws_o + ((size_t)slot * C::kRT + rr) * a.D + ch * 4), v);
          if (ch == 0) __stcg(a.ws_ml + (size_t)slot * C::kRT + rr, make_float2(M, L));
        }
      }
      if (c0 != c1) {
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
                const size_t row = (size_t)unit_slot(min(cc + k, c1), sp.per, w.u0) * C::kRT + rr;
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
      pm_step<C::kRT>(a, w);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && bars->abort) set_dev_status(a.dev_status, TV_DEV_TIMEOUT);
}

// ---- host side

static size_t pm_rows(int G, int N) { return (size_t)2 * kPagedMaxCtas * kPagedMaxSms * (G * N <= 16 ? 16 : 32); }

size_t paged_mma_ws(int Hq, int Hkv, int D, int N) {
  const size_t rows = pm_rows(Hq / Hkv, N);
  return kPagedCntBytes + rows * 8 + rows * D * 4;
}

template <int kD, int kMT, bool kCap>
static cudaError_t launch_pm(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, cudaStream_t stream) {
  using C = PmCfg<kD, kMT>;
  cudaError_t e = cudaFuncSetAttribute(paged_mma_kernel<kD, kMT, kCap>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_mma_kernel<kD, kMT, kCap>, dim3((unsigned)(paged_grid_sms() * C::kCtas)), dim3(C::kThreads),
                    C::kSmem, stream, nullptr, 0, mk, mv, a);
}

template <int kD>
static cudaError_t launch_pm_d(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a, cudaStream_t stream) {
  const bool cap = a.cap > 0.f;
  if (a.G * a.N <= 16)
    return cap ? launch_pm<kD, 1, true>(mk, mv, a, stream) : launch_pm<kD, 1, false>(mk, mv, a, stream);
  return cap ? launch_pm<kD, 2, true>(mk, mv, a, stream) : launch_pm<kD, 2, false>(mk, mv, a, stream);
}

cudaError_t launch_paged_mma(PagedAttn a, char* ws, cudaStream_t stream) {
  a.cnt = reinterpret_cast<unsigned*>(ws);
  a.ws_ml = reinterpret_cast<float2*>(ws + kPagedCntBytes);
  a.ws_o = reinterpret_cast<float*>(ws + kPagedCntBytes + pm_rows(a.G, a.N) * 8);
  const int ps = 1 << a.page_shift, box = min(ps, kPmKeys);
  CUtensorMap mk, mv;
  if (!paged_tmap(&mk, a.k, a.D, ps, (long long)a.num_pages * a.Hkv, box) ||
      !paged_tmap(&mv, a.v, a.D, ps, (long long)a.num_pages * a.Hkv, box))
    return cudaErrorInvalidValue;
  if (a.D <= 64) return launch_pm_d<64>(mk, mv, a, stream);
  if (a.D <= 128) return launch_pm_d<128>(mk, mv, a, stream);
  return launch_pm_d<256>(mk, mv, a, stream);
}

}  // namespace tv
