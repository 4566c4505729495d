// Attention of few new rows (single tokens, short chunks, small trees) over a paged fp32 KV
// cache, on CUDA cores (more rows: paged_f32.cu).
//
//   out[b,h,i,:] = sum_j softmax_j(z_ij) v_j,  z = scale q_i . k_j, or cap tanh(scale q_i . k_j / cap)
//
// over the keys j that row i sees: the committed rows 0..P_b-1 and, of the new rows, 0..i
// (causal) or i and its ancestors (tree), less those `window` or more positions back.
//
// One CTA takes RT = 8 kRPW query rows of a KV head (row r is head r % G of node r / G) and
// walks its range of 32-key tiles, which cp.async brings into three buffers.  A warp
// owns kRPW rows: lane j scores key j against each (K rows padded by 16 bytes, so the 8
// lanes of a 128-bit phase hit different banks), the warp keeps the running maximum and sum
// of each row in 32 bits, and P goes through shared memory so that four keys' weights
// come in one broadcast load.  The units' tiles are divided equally over the CTAs
// (paged.cuh); the CTA that finishes a cut unit last merges its parts in CTA order, so
// results do not depend on which one that is.
#include "paged.cuh"

namespace tv {

constexpr int kPsWarps = 8;
constexpr int kPsKeys = 32;
constexpr int kPsStages = 3;  // K and V tiles in shared memory: two on their way while one is used
// paged_rows_kernel: a unit's set-up and end count as 4 tiles, cuts less than 8 from an edge move to
// it.  0 and 0 / 8 and 4: 23 sequences of 631 to 1262 tokens 21.5 / 18.5 us, one of 2048 (8 heads) 15.1 / 11.3.
constexpr int kPrTol = 8, kPrFix = 4;
constexpr int kPsMerge = 4;  // parts whose loads are in flight together

template <int kDPL, int kRPW>
struct PsSmem {
  static constexpr int kD = kDPL * 32;
  static constexpr int kRT = kPsWarps * kRPW;
  static constexpr int kStride = kD + 4;  // K row in smem, elements
  static constexpr int kOffV = kPsStages * kPsKeys * kStride * 4;
  static constexpr int kOffQ = kOffV + kPsStages * kPsKeys * kD * 4;
  static constexpr int kOffP = kOffQ + kRT * kD * 4;
  static constexpr int kOffVis = kOffP + kRT * kPsKeys * 4;
  static constexpr int kOffPar = kOffVis + kRT * (kMaxNodes / 32) * 4;
  static constexpr int kBytes = kOffPar + kMaxNodes * 4;
  // CTAs that an SM's 228 KB hold, with 1 KB each of the system's: the grid has no more, so that a share
  // of the device keeps to its SMs
  static constexpr int kStatic = 4608;
  static constexpr int kPerSm = kDPL <= 4 && 2 * (kBytes + kStatic + 1024) <= 228 * 1024 ? 2 : 1;
};

// Output of a unit's rows from its parts, in CTA order; a warp per row.
template <int kDPL>
__device__ __forceinline__ void ps_merge(const PagedAttn& a, int b, int hk, int rt, int RT, int rows, int n_act,
                                         long long c0, long long c1, long long per, long long u0) {
  constexpr int kD = kDPL * 32;
  const int lane = threadIdx.x & 31;
  float* out = reinterpret_cast<float*>(a.out);
  for (int rr = threadIdx.x >> 5; rr < rows; rr += kPsWarps) {
    const int r = rt * RT + rr, i = r / a.G, g = r % a.G;
    if (i >= n_act) continue;
    // one pass in batches of independent loads, with a running maximum
    float M = -INFINITY, L = 0.f, o[kDPL];
#pragma unroll
    for (int u = 0; u < kDPL; ++u) o[u] = 0.f;
    for (long long cc = c0; cc <= c1; cc += kPsMerge) {
      float2 ml[kPsMerge];
      float x[kPsMerge][kDPL];
#pragma unroll
      for (int k = 0; k < kPsMerge; ++k) {
        const size_t row = (size_t)unit_slot(min(cc + k, c1), per, u0) * RT + rr;
        ml[k] = __ldcg(&a.ws_ml[row]);
#pragma unroll
        for (int u = 0; u < kDPL; ++u) x[k][u] = __ldcg(&a.ws_o[row * kD + lane + 32 * u]);
        if (cc + k > c1) ml[k].x = -INFINITY;
      }
      float Mn = M;
#pragma unroll
      for (int k = 0; k < kPsMerge; ++k) Mn = fmaxf(Mn, ml[k].x);
      if (Mn == -INFINITY) continue;
      const float f0 = expf(M - Mn);
      M = Mn;
      L *= f0;
#pragma unroll
      for (int u = 0; u < kDPL; ++u) o[u] *= f0;
#pragma unroll
      for (int k = 0; k < kPsMerge; ++k) {
        if (ml[k].x == -INFINITY) continue;
        const float f = expf(ml[k].x - M);
        L = fmaf(f, ml[k].y, L);
#pragma unroll
        for (int u = 0; u < kDPL; ++u) o[u] = fmaf(f, x[k][u], o[u]);
      }
    }
    const size_t off = (((size_t)b * a.Hq + hk * a.G + g) * a.N + i) * kD;
#pragma unroll
    for (int u = 0; u < kDPL; ++u) out[off + lane + 32 * u] = o[u] / L;
  }
}

template <int kDPL, int kRPW>
__global__ void __launch_bounds__(kPsWarps * 32, PsSmem<kDPL, kRPW>::kPerSm) paged_simt_kernel(PagedAttn a) {
  using S = PsSmem<kDPL, kRPW>;
  constexpr int kD = S::kD, kRT = S::kRT, kVec = 4;
  extern __shared__ __align__(16) unsigned char ps_smem[];
  float* s_k = reinterpret_cast<float*>(ps_smem);
  float* s_v = reinterpret_cast<float*>(ps_smem + S::kOffV);
  float* s_q = reinterpret_cast<float*>(ps_smem + S::kOffQ);
  float* s_p = reinterpret_cast<float*>(ps_smem + S::kOffP);
  uint32_t(*s_vis)[kMaxNodes / 32] = reinterpret_cast<uint32_t(*)[kMaxNodes / 32]>(ps_smem + S::kOffVis);
  int* s_par = reinterpret_cast<int*>(ps_smem + S::kOffPar);
  __shared__ unsigned long long s_red[kPagedRed];
  __shared__ int s_first_pad, s_last, s_depth[kRT], s_page[4][kPsKeys / 8];
  static_assert(sizeof(s_red) + sizeof(s_depth) + sizeof(s_page) + 8 <= S::kStatic, "static arrays");
  const int box_shift = min(a.page_shift, 5), pages_tile = kPsKeys >> box_shift;  // a tile's row pieces, each in one page
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* q = reinterpret_cast<const float*>(a.q);
  float* out = reinterpret_cast<float*>(a.out);

  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const PagedSpan sp = paged_span(a, kRT, kPsKeys, 1, s_red);
  UnitWalk w = unit_walk(sp);
  int tree = -1, n_act = 0;
  while (unit_next(a, w, kRT, kPsKeys)) {
    const int b = w.b, hk = w.hk, rt = w.rt, P = w.P, n = w.n, t0 = w.t0, t1 = w.t1;
    const long long u0 = w.u0;
    const int32_t* table = a.table + (size_t)b * a.max_pages;
    if (tree != b) n_act = n;
    if (a.parent && tree != b) {
      // the tree, checked; its rows past the first padding row are inactive
      __syncthreads();
      if (threadIdx.x == 0) s_first_pad = n;
      __syncthreads();
      int wrong = 0;
      for (int t = threadIdx.x; t < n; t += blockDim.x) {
        const int p = a.parent[(size_t)b * a.N + t];
        const bool prev_pad = t >= 2 && a.parent[(size_t)b * a.N + t - 1] == -1;
        const bool ok = t == 0 ? p == -1 : (p == -1 || (p >= 0 && p < t && !prev_pad));
        if (!ok) wrong = 1;
        s_par[t] = ok ? p : -1;
        if (t > 0 && p == -1) atomicMin(&s_first_pad, t);
      }
      if (wrong) set_dev_status(a.dev_status, TV_DEV_BAD_TREE);
      __syncthreads();
      n_act = s_first_pad;
    }
    tree = b;
    const int rows = unit_rows(a, n, rt, kRT);
    const int lo = unit_lo(a, P, rt, kRT), tile0 = lo / kPsKeys;
    const int hi = min(P + n_act, P + (rt * kRT + rows - 1) / a.G + 1);
    // ---- rows: query, depth and the tree nodes each sees
    __syncthreads();
    for (int rr = warp; rr < kRT; rr += kPsWarps) {
      const int r = rt * kRT + rr, i = r / a.G, g = r % a.G;
      const bool live = rr < rows && i < n_act;
      const size_t qoff = (((size_t)b * a.Hq + hk * a.G + g) * a.N + i) * kD;
      for (int d = lane; d < kD; d += 32) s_q[rr * kD + d] = live ? q[qoff + d] * a.scale : 0.f;
      if (!a.parent) {
        if (lane == 0) s_depth[rr] = i;
        continue;
      }
      for (int w = lane; w < kMaxNodes / 32; w += 32) s_vis[rr][w] = 0u;
      __syncwarp();
      if (lane == 0) {
        int depth = 0;
        for (int at = live ? i : -1; at >= 0; at = s_par[at], ++depth)  // parents fall: ends within n steps
          if (a.window <= 0 || depth < a.window) s_vis[rr][at >> 5] |= 1u << (at & 31);
        s_depth[rr] = max(0, depth - 1);
      }
    }
    float m[kRPW], l[kRPW], acc[kRPW][kDPL];
#pragma unroll
    for (int rw = 0; rw < kRPW; ++rw) {
      m[rw] = -INFINITY;
      l[rw] = 0.f;
#pragma unroll
      for (int t = 0; t < kDPL; ++t) acc[rw][t] = 0.f;
    }
    // rows [lo, hi) of the tile; others (pages past the end, rows behind the window, whose
    // contents may be anything) read as zero
    auto page_of = [&](int t) -> int {
      const int j = (tile0 + t) * kPsKeys + ((int)threadIdx.x << box_shift);
      if ((int)threadIdx.x >= pages_tile || t >= t1 || j >= hi || j + (1 << box_shift) <= lo) return -1;
      const int page = table[j >> a.page_shift];
      if (page >= 0 && page < a.num_pages) return page;
      set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
      return -1;
    };
    auto load_tile = [&](int t, int buf) {
      if (t >= t1) {  // an empty group keeps the count
        asm volatile("cp.async.commit_group;" ::: "memory");
        return;
      }
      constexpr int kChunks = kD / kVec;
      for (int e = threadIdx.x; e < kPsKeys * kChunks; e += blockDim.x) {
        const int jj = e / kChunks, ch = e - jj * kChunks;
        const int j = (tile0 + t) * kPsKeys + jj;
        float* dk = s_k + (buf * kPsKeys + jj) * S::kStride + ch * kVec;
        float* dv = s_v + (buf * kPsKeys + jj) * kD + ch * kVec;
        const int page = j >= lo && j < hi ? s_page[t & 3][jj >> box_shift] : -1;
        if (page >= 0) {
          const size_t off =
              ((((size_t)page * a.Hkv + hk) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * kD + ch * kVec;
          cp_async16(dk, reinterpret_cast<const float*>(a.k) + off);
          cp_async16(dv, reinterpret_cast<const float*>(a.v) + off);
        } else {
          *reinterpret_cast<uint4*>(dk) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(dv) = make_uint4(0, 0, 0, 0);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if ((int)threadIdx.x < pages_tile) {
      for (int u = 0; u < 3; ++u) s_page[(t0 + u) & 3][threadIdx.x] = page_of(t0 + u);
    }
    __syncthreads();
    load_tile(t0, 0);
    load_tile(t0 + 1, 1);
    for (int t = t0; t < t1; ++t) {
      const int buf = (t - t0) % kPsStages;
      load_tile(t + 2, (t + 2 - t0) % kPsStages);
      const int ahead = page_of(t + 3);
      asm volatile("cp.async.wait_group 2;" ::: "memory");
      __syncthreads();
      if ((int)threadIdx.x < pages_tile) s_page[(t + 3) & 3][threadIdx.x] = ahead;
      const int j = (tile0 + t) * kPsKeys + lane;
      float4 part[kRPW];  // four chains
#pragma unroll
      for (int rw = 0; rw < kRPW; ++rw) part[rw] = make_float4(0.f, 0.f, 0.f, 0.f);
      const float* kr = s_k + (buf * kPsKeys + lane) * S::kStride;
#pragma unroll 8
      for (int d = 0; d < kD; d += kVec) {
        const float4 kf = *reinterpret_cast<const float4*>(kr + d);
#pragma unroll
        for (int rw = 0; rw < kRPW; ++rw) {
          const float4 qf = *reinterpret_cast<const float4*>(s_q + (warp * kRPW + rw) * kD + d);
          part[rw].x = fmaf(qf.x, kf.x, part[rw].x);
          part[rw].y = fmaf(qf.y, kf.y, part[rw].y);
          part[rw].z = fmaf(qf.z, kf.z, part[rw].z);
          part[rw].w = fmaf(qf.w, kf.w, part[rw].w);
        }
      }
#pragma unroll
      for (int rw = 0; rw < kRPW; ++rw) {
        const int rr = warp * kRPW + rw, i = (rt * kRT + rr) / a.G;
        bool vis = rr < rows && i < n_act && j < hi;
        if (j < P) {
          vis = vis && (a.window <= 0 || P - j + s_depth[rr] < a.window);
        } else if (vis) {
          const int t_new = j - P;
          vis = a.parent ? (s_vis[rr][t_new >> 5] >> (t_new & 31)) & 1u
                         : t_new <= i && (a.window <= 0 || i - t_new < a.window);
        }
        float z = (part[rw].x + part[rw].y) + (part[rw].z + part[rw].w);
        // expf of a difference, not 2^(z log2 e - m): the product's rounding would cost |z| 2^-24
        if (a.cap > 0.f) z = a.cap * tanh_f32(z / a.cap);
        z = vis ? z : -INFINITY;
        const float mt = warp_max(z);
        float p = 0.f;
        if (mt != -INFINITY) {
          const float mnew = fmaxf(m[rw], mt);
          const float corr = expf(m[rw] - mnew);
          p = expf(z - mnew);
          l[rw] = l[rw] * corr + warp_sum(p);
#pragma unroll
          for (int u = 0; u < kDPL; ++u) acc[rw][u] *= corr;
          m[rw] = mnew;
        }
        s_p[rr * kPsKeys + lane] = p;
      }
      __syncwarp();
#pragma unroll 2
      for (int jj = 0; jj < kPsKeys; jj += 4) {
        float4 pf[kRPW];
#pragma unroll
        for (int rw = 0; rw < kRPW; ++rw)
          pf[rw] = *reinterpret_cast<const float4*>(s_p + (warp * kRPW + rw) * kPsKeys + jj);
#pragma unroll
        for (int u = 0; u < kDPL; ++u) {
          const float* vr = s_v + (buf * kPsKeys + jj) * kD + lane + 32 * u;
          const float v0 = vr[0], v1 = vr[kD], v2 = vr[2 * kD], v3 = vr[3 * kD];
#pragma unroll
          for (int rw = 0; rw < kRPW; ++rw)
            acc[rw][u] = fmaf(pf[rw].w, v3, fmaf(pf[rw].z, v2, fmaf(pf[rw].y, v1, fmaf(pf[rw].x, v0, acc[rw][u]))));
        }
      }
      __syncthreads();
    }
    // ---- write the unit, or this CTA's part of it
    const long long c0 = u0 / sp.per, c1 = (w.u1 - 1) / sp.per;
    const int slot = unit_slot(blockIdx.x, sp.per, u0);
#pragma unroll
    for (int rw = 0; rw < kRPW; ++rw) {
      const int rr = warp * kRPW + rw, r = rt * kRT + rr, i = r / a.G, g = r % a.G;
      if (c0 == c1) {
        if (rr >= rows || i >= n_act) continue;
        const size_t off = (((size_t)b * a.Hq + hk * a.G + g) * a.N + i) * kD;
        const float inv = 1.f / l[rw];
#pragma unroll
        for (int u = 0; u < kDPL; ++u) out[off + lane + 32 * u] = acc[rw][u] * inv;
      } else {
        const size_t row = (size_t)slot * kRT + rr;
        if (lane == 0) a.ws_ml[row] = make_float2(m[rw], l[rw]);
#pragma unroll
        for (int u = 0; u < kDPL; ++u) a.ws_o[row * kD + lane + 32 * u] = acc[rw][u];
      }
    }
    if (c0 == c1) continue;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      s_last = ptx::atom_add_acq_rel_gpu(&a.cnt[c0], 1u) == (unsigned)(c1 - c0);
      if (s_last) a.cnt[c0] = 0u;
      __threadfence();
    }
    __syncthreads();
    if (!s_last) continue;
    ps_merge<kDPL>(a, b, hk, rt, kRT, rows, n_act, c0, c1, sp.per, u0);
  }
}

// ---- at most four query rows of a KV head: the keys, not the rows, spread over the warps
//
// A step is 32 keys a tile, one for each group of 8 lanes of the CTA: the group holds the key's K and V
// rows in registers, 16 bytes a lane and chunk, straight from global memory, adds its lanes'
// products by three shuffles, and keeps its own running maximum, sum and weighted sum of V
// for each row.  The loads of kU tiles are in flight at once.  The groups' results meet by
// shuffles, the warps' in shared memory, in a fixed order, when the piece ends.  A row a warp, as
// above, leaves most warps without work here: 32 sequences of 4000 to 8000 tokens, 8 heads of 128,
// one row each 583 us that way and 234 this (6.8 TB/s, the copy rate); 64 of them with four rows
// a head 1151 and 680 (4.7 TB/s: at 255 registers one CTA an SM with two tiles in flight; two CTAs
// with one tile each 723).  Eight rows, 32 sequences of 2000 to 4000: a row a warp 311, this 433.
template <int kDPL, int kR>
struct PrCfg {
  static constexpr int kD = kDPL * 32;
  static constexpr int kU = kDPL * kR <= 8 && kDPL <= 4 ? 4 : kDPL * kR <= 24 ? 2 : 1;  // what 255 registers hold
  static constexpr int kOffMl = kPsWarps * kR * kD * 4;
  static constexpr int kOffQ = kOffMl + kPsWarps * kR * 8;
  static constexpr int kBytes = kOffQ + kR * kD * 4;
};

template <int kDPL, int kR>
__global__ void __launch_bounds__(kPsWarps * 32, 1) paged_rows_kernel(PagedAttn a) {
  using S = PrCfg<kDPL, kR>;
  constexpr int kD = S::kD, kU = S::kU;
  extern __shared__ __align__(16) unsigned char ps_smem[];
  float* s_o = reinterpret_cast<float*>(ps_smem);
  float2* s_ml = reinterpret_cast<float2*>(ps_smem + S::kOffMl);
  float* s_q = reinterpret_cast<float*>(ps_smem + S::kOffQ);
  __shared__ unsigned long long s_red[kPagedRed];
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, key = warp * 4 + (lane >> 3), gl = lane & 7;
  const float* q = reinterpret_cast<const float*>(a.q);
  float* out = reinterpret_cast<float*>(a.out);

  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const PagedSpan sp = paged_span(a, kR, kPsKeys, 1, s_red, kPrTol, kPrFix);
  UnitWalk w = unit_walk(sp);
  while (unit_next(a, w, kR, kPsKeys)) {
    const int b = w.b, hk = w.hk, P = w.P, n = w.n, t0 = w.t0, t1 = w.t1;
    const int32_t* table = a.table + (size_t)b * a.max_pages;
    // the rows: whether each is one, its first visible key, and the new rows it sees as bits
    int n_act = n, par[kR];
    if (a.parent) {
      bool wrong = false;
#pragma unroll
      for (int t = kR - 1; t >= 0; --t) {
        const int p = t < n ? a.parent[(size_t)b * a.N + t] : 0;
        const bool prev_pad = t >= 2 && t < n && a.parent[(size_t)b * a.N + t - 1] == -1;
        const bool fits = t >= n || (t == 0 ? p == -1 : p == -1 || (p >= 0 && p < t && !prev_pad));
        wrong = wrong || !fits;
        par[t] = fits ? p : -1;
        if (t > 0 && t < n && p == -1) n_act = t;
      }
      if (wrong && threadIdx.x == 0) set_dev_status(a.dev_status, TV_DEV_BAD_TREE);
    }
    const int rows = n * a.G;
    bool live[kR];
    int wlo[kR];
    unsigned fresh[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int i = r / a.G;
      live[r] = r < rows && i < n_act;
      int depth = i;
      fresh[r] = 0;
      if (a.parent) {
        depth = -1;
        int at = i;
#pragma unroll
        for (int k = 0; k < kR; ++k)
          if (at >= 0) {
            ++depth;
            if (a.window <= 0 || depth < a.window) fresh[r] |= 1u << at;
            int up = -1;
#pragma unroll
            for (int c = 0; c < kR; ++c)
              if (c == at) up = par[c];
            at = up;
          }
      } else {
#pragma unroll
        for (int t = 0; t < kR; ++t)
          if (t <= i && (a.window <= 0 || i - t < a.window)) fresh[r] |= 1u << t;
      }
      wlo[r] = a.window > 0 ? P + depth - a.window + 1 : 0;
    }
    const int lo = unit_lo(a, P, 0, kR), hi = P + n_act, tile0 = lo / kPsKeys;
    __syncthreads();  // the piece before's reads of s_q and s_o
    for (int e = threadIdx.x; e < kR * kD; e += blockDim.x) {
      const int r = e / kD, i = r / a.G, g = r % a.G;
      s_q[e] = r < rows && i < n_act ? q[(((size_t)b * a.Hq + hk * a.G + g) * a.N + i) * kD + e % kD] * a.scale : 0.f;
    }
    __syncthreads();
    float m[kR], l[kR];
    float4 acc[kR][kDPL];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < kDPL; ++c) acc[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // this group's key of tile t, and its table entry (read a step ahead, checked when it is used)
    auto needed = [&](int t) -> bool {
      const int j = (tile0 + t) * kPsKeys + key;
      return t < t1 && j >= lo && j < hi;
    };
    auto entry = [&](int t) -> int { return needed(t) ? table[((tile0 + t) * kPsKeys + key) >> a.page_shift] : -1; };
    int page[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) page[u] = entry(t0 + u);
    for (int t = t0; t < t1; t += kU) {
      float4 kf[kU][kDPL], vf[kU][kDPL];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int j = (tile0 + t + u) * kPsKeys + key;
        const bool have = page[u] >= 0 && page[u] < a.num_pages;
        if (needed(t + u) && !have) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
        const size_t off =
            ((((size_t)page[u] * a.Hkv + hk) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * (kD / 4) + gl;
#pragma unroll
        for (int c = 0; c < kDPL; ++c) {
          kf[u][c] = vf[u][c] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (have) {
            kf[u][c] = __ldcg(reinterpret_cast<const float4*>(a.k) + off + 8 * c);
            vf[u][c] = __ldcg(reinterpret_cast<const float4*>(a.v) + off + 8 * c);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) page[u] = entry(t + kU + u);
      float z[kU][kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float4 part[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) part[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kDPL; ++c) {
          const float4 qf = *reinterpret_cast<const float4*>(s_q + r * kD + (gl + 8 * c) * 4);
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            part[u].x = fmaf(qf.x, kf[u][c].x, part[u].x);
            part[u].y = fmaf(qf.y, kf[u][c].y, part[u].y);
            part[u].z = fmaf(qf.z, kf[u][c].z, part[u].z);
            part[u].w = fmaf(qf.w, kf[u][c].w, part[u].w);
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) z[u][r] = (part[u].x + part[u].y) + (part[u].z + part[u].w);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) z[u][r] += __shfl_xor_sync(0xffffffffu, z[u][r], o);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float mt = m[r];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int j = (tile0 + t + u) * kPsKeys + key;
          if (a.cap > 0.f) z[u][r] = a.cap * tanh_f32(z[u][r] / a.cap);
          const bool vis = live[r] && t + u < t1 && j < hi && (j < P ? j >= wlo[r] : (fresh[r] >> (j - P)) & 1u);
          if (!vis) z[u][r] = -INFINITY;
          mt = fmaxf(mt, z[u][r]);
        }
        if (mt == -INFINITY) continue;
        // expf of a difference, not 2^(z log2 e - m): the product's rounding would cost |z| 2^-24
        const float corr = expf(m[r] - mt);
        m[r] = mt;
        l[r] *= corr;
#pragma unroll
        for (int c = 0; c < kDPL; ++c)
          acc[r][c] = make_float4(acc[r][c].x * corr, acc[r][c].y * corr, acc[r][c].z * corr, acc[r][c].w * corr);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const float p = expf(z[u][r] - mt);
          l[r] += p;
#pragma unroll
          for (int c = 0; c < kDPL; ++c) {
            acc[r][c].x = fmaf(p, vf[u][c].x, acc[r][c].x);
            acc[r][c].y = fmaf(p, vf[u][c].y, acc[r][c].y);
            acc[r][c].z = fmaf(p, vf[u][c].z, acc[r][c].z);
            acc[r][c].w = fmaf(p, vf[u][c].w, acc[r][c].w);
          }
        }
      }
    }
    // ---- the warp's four groups, then the eight warps
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      float M = m[r];
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
      const float f = m[r] == -INFINITY ? 0.f : expf(m[r] - M);
      auto over = [&](float x) -> float {
        x *= f;
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        return x + __shfl_xor_sync(0xffffffffu, x, 16);
      };
      const float L = over(l[r]);
      if (lane == 0) s_ml[warp * kR + r] = make_float2(M, L);
#pragma unroll
      for (int c = 0; c < kDPL; ++c) {
        const float4 o = make_float4(over(acc[r][c].x), over(acc[r][c].y), over(acc[r][c].z), over(acc[r][c].w));
        if (lane < 8) *reinterpret_cast<float4*>(s_o + (warp * kR + r) * kD + (gl + 8 * c) * 4) = o;
      }
    }
    __syncthreads();
    const auto [c0, c1] = unit_ctas(w);
    const int slot = unit_slot(blockIdx.x, sp.per, w.u0);
    for (int e = threadIdx.x; e < kR * kD; e += blockDim.x) {
      const int r = e / kD, i = r / a.G, g = r % a.G;
      if (r >= rows || i >= n_act) continue;
      float M = -INFINITY, L = 0.f, o = 0.f;
#pragma unroll
      for (int k = 0; k < kPsWarps; ++k) M = fmaxf(M, s_ml[k * kR + r].x);
#pragma unroll
      for (int k = 0; k < kPsWarps; ++k) {
        const float2 ml = s_ml[k * kR + r];
        if (ml.x == -INFINITY) continue;
        const float f = expf(ml.x - M);
        L = fmaf(f, ml.y, L);
        o = fmaf(f, s_o[(k * kR + r) * kD + e % kD], o);
      }
      if (c1 <= c0) {
        out[(((size_t)b * a.Hq + hk * a.G + g) * a.N + i) * kD + e % kD] = o / L;
      } else {
        const size_t row = (size_t)slot * kR + r;
        __stcg(&a.ws_o[row * kD + e % kD], o);
        if (e % kD == 0) __stcg(&a.ws_ml[row], make_float2(M, L));
      }
    }
    if (c1 <= c0) continue;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      s_last = ptx::atom_add_acq_rel_gpu(&a.cnt[c0], 1u) == (unsigned)(c1 - c0);
      if (s_last) a.cnt[c0] = 0u;
      __threadfence();
    }
    __syncthreads();
    if (s_last) ps_merge<kDPL>(a, b, hk, 0, kR, rows, n_act, c0, c1, sp.per, w.u0);
  }
}

// ---- host side

// counters, (m, l) and O of two partial units per CTA of the largest grid
constexpr size_t kPsRows = (size_t)2 * kPagedMaxCtas * kPagedMaxSms * kPsWarps * 2;

PagedWs paged_simt_ws(int D) {
  const size_t n = kPagedCntBytes + kPsRows * 8 + kPsRows * D * 4;
  return {n, n};
}

template <int kDPL, int kRPW>
static cudaError_t launch_ps(PagedAttn a, char* ws, cudaStream_t stream) {
  using S = PsSmem<kDPL, kRPW>;
  cudaError_t e = cudaFuncSetAttribute(paged_simt_kernel<kDPL, kRPW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       S::kBytes);
  if (e != cudaSuccess) return e;
  a.cnt = reinterpret_cast<unsigned*>(ws);
  a.ws_ml = reinterpret_cast<float2*>(ws + kPagedCntBytes);
  a.ws_o = reinterpret_cast<float*>(ws + kPagedCntBytes + kPsRows * 8);
  return launch_pdl(paged_simt_kernel<kDPL, kRPW>, dim3((unsigned)(a.sms * S::kPerSm)),
                    dim3(kPsWarps * 32), S::kBytes, stream, nullptr, 0, a);
}

template <int kDPL, int kR>
static cudaError_t launch_pr(PagedAttn a, char* ws, cudaStream_t stream) {
  using S = PrCfg<kDPL, kR>;
  cudaError_t e = cudaFuncSetAttribute(paged_rows_kernel<kDPL, kR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       S::kBytes);
  if (e != cudaSuccess) return e;
  a.cnt = reinterpret_cast<unsigned*>(ws);
  a.ws_ml = reinterpret_cast<float2*>(ws + kPagedCntBytes);
  a.ws_o = reinterpret_cast<float*>(ws + kPagedCntBytes + kPsRows * 8);
  return launch_pdl(paged_rows_kernel<kDPL, kR>, dim3((unsigned)a.sms), dim3(kPsWarps * 32), S::kBytes,
                    stream, nullptr, 0, a);
}

template <int kR>
static cudaError_t launch_pr_d(const PagedAttn& a, char* ws, cudaStream_t stream) {
  switch (a.D / 32) {
    case 1:
      return launch_pr<1, kR>(a, ws, stream);
    case 2:
      return launch_pr<2, kR>(a, ws, stream);
    case 3:
      return launch_pr<3, kR>(a, ws, stream);
    case 4:
      return launch_pr<4, kR>(a, ws, stream);
    case 5:
      return launch_pr<5, kR>(a, ws, stream);
    case 6:
      return launch_pr<6, kR>(a, ws, stream);
    case 7:
      return launch_pr<7, kR>(a, ws, stream);
    case 8:
      return launch_pr<8, kR>(a, ws, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

template <int kRPW>
static cudaError_t launch_ps_d(const PagedAttn& a, char* ws, cudaStream_t stream) {
  switch (a.D / 32) {
    case 1:
      return launch_ps<1, kRPW>(a, ws, stream);
    case 2:
      return launch_ps<2, kRPW>(a, ws, stream);
    case 3:
      return launch_ps<3, kRPW>(a, ws, stream);
    case 4:
      return launch_ps<4, kRPW>(a, ws, stream);
    case 5:
      return launch_ps<5, kRPW>(a, ws, stream);
    case 6:
      return launch_ps<6, kRPW>(a, ws, stream);
    case 7:
      return launch_ps<7, kRPW>(a, ws, stream);
    case 8:
      return launch_ps<8, kRPW>(a, ws, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

cudaError_t launch_paged_simt(PagedAttn a, char* ws, cudaStream_t stream) {
  const int rows = a.G * a.N;  // up to four: keys spread over the warps (both sides measured above)
  if (rows == 1) return launch_pr_d<1>(a, ws, stream);
  if (rows == 2) return launch_pr_d<2>(a, ws, stream);
  if (rows <= 4) return launch_pr_d<4>(a, ws, stream);
  // up to eight: one a warp, so that a KV head's rows spread over a CTA's warps
  return a.G * a.N <= kPsWarps ? launch_ps_d<1>(a, ws, stream) : launch_ps_d<2>(a, ws, stream);
}

}  // namespace tv
