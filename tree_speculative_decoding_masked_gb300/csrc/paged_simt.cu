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
#include "paged_rows.cuh"

namespace tv {

constexpr int kPsStages = 3;  // K and V tiles in shared memory: two on their way while one is used

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

// ---- host side

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
  // up to four: keys spread over the warps (both sides measured there)
  if (a.G * a.N <= 4) return launch_paged_rows<false>(a, ws, stream);
  // up to eight: one a warp, so that a KV head's rows spread over a CTA's warps
  return a.G * a.N <= kPsWarps ? launch_ps_d<1>(a, ws, stream) : launch_ps_d<2>(a, ws, stream);
}

}  // namespace tv
