// Attention of at most four query rows of a KV head over fp32 or 8-bit pages, in 32 bits: the keys, not the
// rows, are spread over the warps (more rows: paged_simt.cu, paged_f32.cuh).
//
// A step is 32 keys a tile, one for each group of 8 lanes of the CTA: the group holds the key's K and V
// rows in registers, 16 bytes a lane and chunk, straight from global memory, adds its lanes'
// products by three shuffles, and keeps its own running maximum, sum and weighted sum of V
// for each row.  The loads of kU tiles are in flight at once.  The groups' results meet by
// shuffles, the warps' in shared memory, in a fixed order, when the piece ends.  A row a warp, as
// in paged_simt_kernel, leaves most warps without work here: 32 sequences of 4000 to 8000 tokens, 8 heads of 128,
// one row each 583 us that way and 234 this (6.8 TB/s, the copy rate); 64 of them with four rows
// a head 1151 and 680 (4.7 TB/s: at 255 registers one CTA an SM with two tiles in flight; two CTAs
// with one tile each 723).  Eight rows, 32 sequences of 2000 to 4000: a row a warp 311, this 433.
#pragma once

#include <string.h>

#include <type_traits>

#include "paged.cuh"
#include "q8.cuh"

namespace tv {

constexpr int kPsWarps = 8;
constexpr int kPsKeys = 32;
// paged_rows_kernel: a unit's set-up and end count as 4 tiles, cuts less than 8 from an edge move to
// it.  0 and 0 / 8 and 4: 23 sequences of 631 to 1262 tokens 21.5 / 18.5 us, one of 2048 (8 heads) 15.1 / 11.3.
constexpr int kPrTol = 8, kPrFix = 4;
constexpr int kPsMerge = 4;  // parts whose loads are in flight together

// counters, (m, l) and O of two partial units per CTA of the largest grid
constexpr size_t kPsRows = (size_t)2 * kPagedMaxCtas * kPagedMaxSms * kPsWarps * 2;

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

template <int kDPL, int kR>
struct PrCfg {
  static constexpr int kD = kDPL * 32;
  static constexpr int kU = kDPL * kR <= 8 && kDPL <= 4 ? 4 : kDPL * kR <= 24 ? 2 : 1;  // what 255 registers hold
  static constexpr int kUQ8 = kR * kDPL <= 8 ? 8 : kR * kDPL <= 16 ? 4 : 1;
  static constexpr int kOffMl = kPsWarps * kR * kD * 4;
  static constexpr int kOffQ = kOffMl + kPsWarps * kR * 8;
  static constexpr int kBytes = kOffQ + kR * kD * 4;
};

// kQ8: K and V are e4m3 codes with block scales (q8.cuh).  A lane holds kDPL words of four, and turns them into
// numbers where they are used; V's scale multiplies the weight.  32 sequences of 4000 to 8000
// tokens, 8 KV heads of 128, one row each: 142 us (2.5 TB/s; 64 rows a tile, as for many rows, 992), two rows 175,
// four 306: eight warps an SM at up to 255 registers wait for what they turn and multiply.  Half the tiles in flight
// 150, 183 and 430.
template <int kDPL, int kR, bool kQ8>
__global__ void __launch_bounds__(kPsWarps * 32, 1) paged_rows_kernel(PagedAttn a) {
  using S = PrCfg<kDPL, kR>;
  constexpr int kD = S::kD, kU = kQ8 ? S::kUQ8 : S::kU;
  // the lane's words or quads c = 0 .. kDPL - 1 are elements 4 place(c) .. 4 place(c) + 3: codes come kW words a load
  constexpr int kW = !kQ8 ? 1 : kDPL % 4 == 0 ? 4 : kDPL % 2 == 0 ? 2 : 1;
  extern __shared__ __align__(16) unsigned char ps_smem[];
  float* s_o = reinterpret_cast<float*>(ps_smem);
  float2* s_ml = reinterpret_cast<float2*>(ps_smem + S::kOffMl);
  float* s_q = reinterpret_cast<float*>(ps_smem + S::kOffQ);
  __shared__ unsigned long long s_red[kPagedRed];
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, key = warp * 4 + (lane >> 3), gl = lane & 7;
  auto place = [&](int c) -> int { return c / kW * 8 * kW + gl * kW + c % kW; };
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
      using Quad = std::conditional_t<kQ8, uint32_t, float4>;
      Quad kf[kU][kDPL], vf[kU][kDPL];
      unsigned ks[kU], vs[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int j = (tile0 + t + u) * kPsKeys + key;
        const bool have = page[u] >= 0 && page[u] < a.num_pages;
        if (needed(t + u) && !have) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
        const size_t row = (((size_t)page[u] * a.Hkv + hk) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
        if constexpr (kQ8) {
          ks[u] = vs[u] = 127;
#pragma unroll
          for (int c = 0; c < kDPL; ++c) kf[u][c] = vf[u][c] = 0;
          if (have) {
            ks[u] = a.ks[row >> a.block_shift], vs[u] = a.vs[row >> a.block_shift];
            const uint32_t* k = reinterpret_cast<const uint32_t*>(a.k) + row * (kD / 4) + gl * kW;
            const uint32_t* v = reinterpret_cast<const uint32_t*>(a.v) + row * (kD / 4) + gl * kW;
            using Wide = std::conditional_t<kW == 4, uint4, std::conditional_t<kW == 2, uint2, uint32_t>>;
#pragma unroll
            for (int c = 0; c < kDPL; c += kW) {
              const Wide x = __ldcg(reinterpret_cast<const Wide*>(k + 8 * c));
              const Wide y = __ldcg(reinterpret_cast<const Wide*>(v + 8 * c));
              memcpy(&kf[u][c], &x, sizeof(Wide));
              memcpy(&vf[u][c], &y, sizeof(Wide));
            }
          }
        } else {
          const size_t off = row * (kD / 4) + gl;
#pragma unroll
          for (int c = 0; c < kDPL; ++c) {
            kf[u][c] = vf[u][c] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (have) {
              kf[u][c] = __ldcg(reinterpret_cast<const float4*>(a.k) + off + 8 * c);
              vf[u][c] = __ldcg(reinterpret_cast<const float4*>(a.v) + off + 8 * c);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) page[u] = entry(t + kU + u);
      float z[kU][kR];
      auto score = [&](float4& p, const float4& qf, const float4& k) {
        p.x = fmaf(qf.x, k.x, p.x);
        p.y = fmaf(qf.y, k.y, p.y);
        p.z = fmaf(qf.z, k.z, p.z);
        p.w = fmaf(qf.w, k.w, p.w);
      };
      if constexpr (kQ8) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          // numbers, not codes: a large query's products with codes might not fit before the scale
          const float2 scale = make_float2(q8_scale(ks[u]), q8_scale(ks[u]));
          float2 part[kR][2];
#pragma unroll
          for (int r = 0; r < kR; ++r) part[r][0] = part[r][1] = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < kDPL; ++c) {
            const float4 k = q8_quad(kf[u][c]);
            const float2 k0 = __fmul2_rn(make_float2(k.x, k.y), scale), k1 = __fmul2_rn(make_float2(k.z, k.w), scale);
#pragma unroll
            for (int r = 0; r < kR; ++r) {
              const float4 qf = *reinterpret_cast<const float4*>(s_q + r * kD + place(c) * 4);
              part[r][0] = __ffma2_rn(make_float2(qf.x, qf.y), k0, part[r][0]);
              part[r][1] = __ffma2_rn(make_float2(qf.z, qf.w), k1, part[r][1]);
            }
          }
#pragma unroll
          for (int r = 0; r < kR; ++r) z[u][r] = (part[r][0].x + part[r][0].y) + (part[r][1].x + part[r][1].y);
        }
      } else {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          float4 part[kU];
#pragma unroll
          for (int u = 0; u < kU; ++u) part[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int c = 0; c < kDPL; ++c) {
            const float4 qf = *reinterpret_cast<const float4*>(s_q + r * kD + (gl + 8 * c) * 4);
#pragma unroll
            for (int u = 0; u < kU; ++u) score(part[u], qf, kf[u][c]);
          }
#pragma unroll
          for (int u = 0; u < kU; ++u) z[u][r] = (part[u].x + part[u].y) + (part[u].z + part[u].w);
        }
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
          if constexpr (kQ8) {
            z[u][r] = p;
          } else {
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
      if constexpr (kQ8) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const float scale = q8_scale(vs[u]);
          float p[kR];
#pragma unroll
          for (int r = 0; r < kR; ++r) p[r] = z[u][r] == -INFINITY ? 0.f : z[u][r] * scale;  // no row has seen a key yet
#pragma unroll
          for (int c = 0; c < kDPL; ++c) {
            const float4 v = q8_quad(vf[u][c]);
#pragma unroll
            for (int r = 0; r < kR; ++r) {
              const float2 w = make_float2(p[r], p[r]);
              const float2 a0 = __ffma2_rn(w, make_float2(v.x, v.y), make_float2(acc[r][c].x, acc[r][c].y));
              const float2 a1 = __ffma2_rn(w, make_float2(v.z, v.w), make_float2(acc[r][c].z, acc[r][c].w));
              acc[r][c] = make_float4(a0.x, a0.y, a1.x, a1.y);
            }
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
        if (lane < 8) *reinterpret_cast<float4*>(s_o + (warp * kR + r) * kD + place(c) * 4) = o;
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

template <int kDPL, int kR, bool kQ8>
static cudaError_t launch_pr(PagedAttn a, char* ws, cudaStream_t stream) {
  using S = PrCfg<kDPL, kR>;
  cudaError_t e = cudaFuncSetAttribute(paged_rows_kernel<kDPL, kR, kQ8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       S::kBytes);
  if (e != cudaSuccess) return e;
  a.cnt = reinterpret_cast<unsigned*>(ws);
  a.ws_ml = reinterpret_cast<float2*>(ws + kPagedCntBytes);
  a.ws_o = reinterpret_cast<float*>(ws + kPagedCntBytes + kPsRows * 8);
  return launch_pdl(paged_rows_kernel<kDPL, kR, kQ8>, dim3((unsigned)a.sms), dim3(kPsWarps * 32), S::kBytes,
                    stream, nullptr, 0, a);
}

template <int kR, bool kQ8>
static cudaError_t launch_pr_d(const PagedAttn& a, char* ws, cudaStream_t stream) {
  switch (a.D / 32) {
    case 1:
      return launch_pr<1, kR, kQ8>(a, ws, stream);
    case 2:
      return launch_pr<2, kR, kQ8>(a, ws, stream);
    case 3:
      return launch_pr<3, kR, kQ8>(a, ws, stream);
    case 4:
      return launch_pr<4, kR, kQ8>(a, ws, stream);
    case 5:
      return launch_pr<5, kR, kQ8>(a, ws, stream);
    case 6:
      return launch_pr<6, kR, kQ8>(a, ws, stream);
    case 7:
      return launch_pr<7, kR, kQ8>(a, ws, stream);
    case 8:
      return launch_pr<8, kR, kQ8>(a, ws, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

template <bool kQ8>
static cudaError_t launch_paged_rows(const PagedAttn& a, char* ws, cudaStream_t stream) {
  const int rows = a.G * a.N;
  if (rows == 1) return launch_pr_d<1, kQ8>(a, ws, stream);
  if (rows == 2) return launch_pr_d<2, kQ8>(a, ws, stream);
  return launch_pr_d<4, kQ8>(a, ws, stream);
}

}  // namespace tv
