// Attention of many rows over a paged fp32 KV cache on CUDA cores (chunks and trees; few rows:
// paged_simt.cu).  The arithmetic stays fp32 throughout, so the FMA pipes bound it: the tile is
// shaped to feed them from registers.
//
// A CTA takes 64 query rows of a KV head (row r is head r % G of node r / G) against 64-key
// tiles, double-buffered by cp.async (D <= 128).  Thread (tx, ty) of 16 x 16 scores rows
// 4 ty + a against keys tx + 16 b, 64 FMAs for 8 loads of 16 bytes per 4 columns (a warp's loads
// are 2 rows' broadcasts or 16 padded key rows); a row's softmax statistics meet by shuffles
// over its 16 threads; P passes through shared memory, and the thread accumulates columns
// 2 tx + 32 u of its four rows.  Few units run as clusters whose CTAs take equal parts of the
// keys and merge a share of the rows each; more are divided over a persistent grid
// (paged.cuh).  Two 100-node trees, 8 heads of 64, window 1024: 57 -> 38 us against that
// kernel's 32 rows, one row a warp at a time.
#pragma once

#include "paged.cuh"
#include "q8.cuh"

namespace tv {

constexpr int kPfThreads = 256;
constexpr int kPfRows = 64;
constexpr int kPfKeys = 64;
constexpr int kPfMaxSplits = 8;  // portable cluster size
constexpr int kPfMerge = 4;  // parts whose loads are in flight together

template <int kD>
struct PfSmem {
  static constexpr int kBufs = kD <= 128 ? 2 : 1;
  static constexpr int kStride = kD + 4;             // floats of a Q or K row: 16 rows on different banks
  static constexpr int kPStride = kPfKeys + 4;
  static constexpr int kOffK = kPfRows * kStride;
  static constexpr int kOffV = kOffK + kBufs * kPfKeys * kStride;
  static constexpr int kOffP = kOffV + kBufs * kPfKeys * kD;
  static constexpr int kBytes = (kOffP + kPfRows * kPStride) * 4;
};

// kQ8: K and V are e4m3 codes with block scales (q8.cuh), turned into fp32 numbers as they are stored to
// shared memory: a tile's codes wait in registers while the tile before is used.  The multiply-adds bound both alike:
// two 100-node trees, 8 heads over 4 of 64, window 1024, capped, 38.6 us; 8 heads over 8, 1024 rows over 4000, 572
// (fp32 pages 530).  8 rows of 32 sequences over 2000 to 4000 take 490, seven eighths of their tiles being empty.
template <int kD, bool kStream, bool kQ8>
__global__ void __launch_bounds__(kPfThreads, kD <= 64 ? 2 : 1)
    paged_f32_kernel(PagedAttn a, int splits, int row_tiles) {
  using S = PfSmem<kD>;
  constexpr int kU = kD / 32;
  extern __shared__ __align__(16) float pf_smem[];
  float* s_q = pf_smem;
  float* s_k = pf_smem + S::kOffK;
  float* s_v = pf_smem + S::kOffV;
  float* s_p = pf_smem + S::kOffP;
  __shared__ __align__(8) uint32_t s_vis[kPfRows][kMaxNodes / 32];
  unsigned long long* s_red = reinterpret_cast<unsigned long long*>(s_vis);  // before the first unit
  static_assert(sizeof(s_vis) >= kPagedRed * 8, "scratch of the division");
  __shared__ int s_par[kMaxNodes];
  __shared__ int s_lo[kPfRows], s_hi[kPfRows], s_page[2][kPfKeys / 8], s_first_pad, s_last;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const float* q = reinterpret_cast<const float*>(a.q);
  float* out = reinterpret_cast<float*>(a.out);
  constexpr int kC = kQ8 ? (kPfKeys * (kD / 16) + kPfThreads - 1) / kPfThreads : 1;  // 16 codes each
  uint4 k_raw[kC], v_raw[kC];
  float k_scale[kC], v_scale[kC];

  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int pages_tile = max(1, kPfKeys >> a.page_shift);
  const float inv_cap = a.cap > 0.f ? 1.f / a.cap : 0.f;
  const size_t cta = ((size_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  PagedSpan sp{};
  UnitWalk w{};
  if constexpr (kStream) {
    sp = paged_span(a, kPfRows, kPfKeys, 1, s_red);
    __syncthreads();
    w = unit_walk(sp);
  } else {
    // the cluster's unit, and this CTA's part of its tiles
    bool bad = false;
    w.b = blockIdx.z, w.hk = blockIdx.y / row_tiles, w.rt = blockIdx.y % row_tiles;
    w.P = a.prefix_len[w.b];
    w.n = paged_rows(a, w.b, w.P, &bad);
    if (w.n == 0) w.P = 0;
    if (threadIdx.x == 0 && (bad || paged_cut(a, w.b, w.P, w.n))) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
    const int T_u = unit_tiles(a, w.P, w.n, w.rt, kPfRows, kPfKeys), part = blockIdx.x;
    w.t0 = (int)((long long)T_u * part / splits);
    w.t1 = (int)((long long)T_u * (part + 1) / splits);
  }
  int tree = -1, n_act = 0;
  for (bool once = true; kStream ? unit_next(a, w, kPfRows, kPfKeys) : once; once = false) {
    const int b = w.b, hk = w.hk, rt = w.rt, P = w.P, n = w.n, t0 = w.t0, t1 = w.t1;
    const long long u0 = w.u0, u1 = w.u1;
    const int32_t* table = a.table + (size_t)b * a.max_pages;
    if (tree != b) n_act = n;
    if (a.parent && n > 0 && tree != b) {
      __syncthreads();
      if (threadIdx.x == 0) s_first_pad = n;
      __syncthreads();
      int wrong = 0;
      for (int t = threadIdx.x; t < n; t += kPfThreads) {
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
    const int rows = unit_rows(a, n, rt, kPfRows), r0 = rt * kPfRows;
    const int lo = unit_lo(a, P, rt, kPfRows), tile0 = lo / kPfKeys;
    const int hi = min(P + n_act, P + (r0 + rows - 1) / a.G + 1);
    // page of piece `threadIdx.x` of tile t, -1 where no row is needed
    auto page_of = [&](int t) -> int {
      const int j = (tile0 + t) * kPfKeys + ((int)threadIdx.x << min(a.page_shift, 6));
      if ((int)threadIdx.x >= pages_tile || t >= t1 || j >= hi || j + (1 << min(a.page_shift, 6)) <= lo) return -1;
      const int page = table[j >> a.page_shift];
      if (page >= 0 && page < a.num_pages) return page;
      set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
      return -1;
    };
    // rows [lo, hi) of tile t; others (pages past the end, rows behind the window, whose contents
    // may be anything) read as zero
    auto fetch_q8 = [&](int t) {
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int e = c * kPfThreads + threadIdx.x, jj = e / (kD / 16), ch = e - jj * (kD / 16);
        const int j = (tile0 + t) * kPfKeys + jj;
        k_raw[c] = v_raw[c] = make_uint4(0, 0, 0, 0);
        k_scale[c] = v_scale[c] = 0.f;
        const int page = jj < kPfKeys && j >= lo && j < hi ? s_page[t & 1][jj >> min(a.page_shift, 6)] : -1;
        if (page >= 0) {
          const size_t row = (((size_t)page * a.Hkv + hk) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
          k_raw[c] = __ldcg(reinterpret_cast<const uint4*>(a.k) + row * (kD / 16) + ch);
          v_raw[c] = __ldcg(reinterpret_cast<const uint4*>(a.v) + row * (kD / 16) + ch);
          k_scale[c] = q8_scale(a.ks[row >> a.block_shift]);
          v_scale[c] = q8_scale(a.vs[row >> a.block_shift]);
        }
      }
    };
    auto place_q8 = [&](int buf) {
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int e = c * kPfThreads + threadIdx.x, jj = e / (kD / 16), ch = e - jj * (kD / 16);
        if (jj >= kPfKeys) continue;
        float4* dk = reinterpret_cast<float4*>(s_k + (buf * kPfKeys + jj) * S::kStride + ch * 16);
        float4* dv = reinterpret_cast<float4*>(s_v + (buf * kPfKeys + jj) * kD + ch * 16);
        dk[0] = q8_numbers(k_raw[c].x, k_scale[c]), dk[1] = q8_numbers(k_raw[c].y, k_scale[c]);
        dk[2] = q8_numbers(k_raw[c].z, k_scale[c]), dk[3] = q8_numbers(k_raw[c].w, k_scale[c]);
        dv[0] = q8_numbers(v_raw[c].x, v_scale[c]), dv[1] = q8_numbers(v_raw[c].y, v_scale[c]);
        dv[2] = q8_numbers(v_raw[c].z, v_scale[c]), dv[3] = q8_numbers(v_raw[c].w, v_scale[c]);
      }
    };
    auto load_tile = [&](int t, int buf) {
      for (int e = threadIdx.x; e < kPfKeys * (kD / 4); e += kPfThreads) {
        const int jj = e / (kD / 4), ch = e - jj * (kD / 4);
        const int j = (tile0 + t) * kPfKeys + jj;
        float* dk = s_k + (buf * kPfKeys + jj) * S::kStride + ch * 4;
        float* dv = s_v + (buf * kPfKeys + jj) * kD + ch * 4;
        const int page = j >= lo && j < hi ? s_page[t & 1][jj >> min(a.page_shift, 6)] : -1;
        if (page >= 0) {
          const size_t off =
              ((((size_t)page * a.Hkv + hk) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * kD + ch * 4;
          cp_async16(dk, reinterpret_cast<const float*>(a.k) + off);
          cp_async16(dv, reinterpret_cast<const float*>(a.v) + off);
        } else {
          *reinterpret_cast<float4*>(dk) = make_float4(0.f, 0.f, 0.f, 0.f);
          *reinterpret_cast<float4*>(dv) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncthreads();
    // ---- rows: queries, bounds and the tree nodes each sees
    if ((int)threadIdx.x < pages_tile) {
      s_page[t0 & 1][threadIdx.x] = page_of(t0);
      s_page[(t0 + 1) & 1][threadIdx.x] = page_of(t0 + 1);
    }
    for (int e = threadIdx.x; e < kPfRows * (kD / 4); e += kPfThreads) {
      const int rr = e / (kD / 4), ch = e - rr * (kD / 4), i = (r0 + rr) / a.G, g = (r0 + rr) % a.G;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (rr < rows && i < n_act) {
        v = *reinterpret_cast<const float4*>(q + (((size_t)b * a.Hq + hk * a.G + g) * a.N + i) * kD + ch * 4);
        v.x *= a.scale, v.y *= a.scale, v.z *= a.scale, v.w *= a.scale;
      }
      *reinterpret_cast<float4*>(s_q + rr * S::kStride + ch * 4) = v;
    }
    if (threadIdx.x < kPfRows) {
      const int rr = threadIdx.x, i = (r0 + rr) / a.G;
      int wlo = 0, whi = -1;  // what is no row sees nothing
      if (rr < rows && i < n_act) {
        int depth = i;
        whi = a.parent ? P : P + i + 1;
        if (a.parent) {
          depth = -1;
          for (int w = 0; w < (n + 31) / 32; ++w) s_vis[rr][w] = 0u;
          for (int at = i; at >= 0; at = s_par[at]) {  // parents fall: it ends
            ++depth;
            if (a.window <= 0 || depth < a.window) s_vis[rr][at >> 5] |= 1u << (at & 31);
          }
        }
        if (a.window > 0) wlo = P + depth - a.window + 1;
      }
      s_lo[rr] = wlo;
      s_hi[rr] = whi;
    }
    __syncthreads();
    float m[4], l[4], acc[4][kU][2];
    int wlo[4], whi[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      m[x] = -INFINITY;
      l[x] = 0.f;
      wlo[x] = s_lo[ty * 4 + x];
      whi[x] = s_hi[ty * 4 + x];
#pragma unroll
      for (int u = 0; u < kU; ++u) acc[x][u][0] = acc[x][u][1] = 0.f;
    }
    const bool live = (ty & ~1) * 4 < rows;  // some of this warp's eight rows are rows
    if constexpr (kQ8) {
      if (t0 < t1) {
        fetch_q8(t0);
        place_q8(0);
      }
    } else {
      load_tile(t0, 0);
    }
    // the next tile: into the other buffer where there is one, before the warps meet, else behind that
    auto next_q8 = [&](int t, int buf) {
      if (kQ8 && S::kBufs == 2 && t + 1 < t1) place_q8(buf ^ 1);
      __syncthreads();
      if (kQ8 && S::kBufs == 1 && t + 1 < t1) place_q8(0);
    };
    for (int t = t0; t < t1; ++t) {
      const int buf = S::kBufs == 2 ? (t - t0) & 1 : 0;
      int ahead = -1;
      if constexpr (kQ8) {
        if (t + 1 < t1) fetch_q8(t + 1);
        ahead = page_of(t + 2);
      } else if (S::kBufs == 2 && t + 1 < t1) {
        load_tile(t + 1, buf ^ 1);
        ahead = page_of(t + 2);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        ahead = page_of(t + 2);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncthreads();
      if ((int)threadIdx.x < pages_tile) s_page[t & 1][threadIdx.x] = ahead;  // tile t + 2's; t's are used up
      if (!live) {
        next_q8(t, buf);
        if (!kQ8 && S::kBufs == 1 && t + 1 < t1) load_tile(t + 1, 0);
        continue;
      }
      // ---- scores
      float s[4][4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) s[x][y] = 0.f;
      const float* qr = s_q + ty * 4 * S::kStride;
      const float* kr = s_k + (buf * kPfKeys + tx) * S::kStride;
#pragma unroll 4
      for (int d = 0; d < kD; d += 4) {
        float4 qf[4], kf[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) qf[x] = *reinterpret_cast<const float4*>(qr + x * S::kStride + d);
#pragma unroll
        for (int y = 0; y < 4; ++y) kf[y] = *reinterpret_cast<const float4*>(kr + y * 16 * S::kStride + d);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            s[x][y] = fmaf(qf[x].x, kf[y].x, s[x][y]);
            s[x][y] = fmaf(qf[x].y, kf[y].y, s[x][y]);
            s[x][y] = fmaf(qf[x].z, kf[y].z, s[x][y]);
            s[x][y] = fmaf(qf[x].w, kf[y].w, s[x][y]);
          }
      }
      // ---- weights, against a running reference that moves when a score exceeds it by 5.5 (e^5.5
      // = 245): the maximum over a row's 16 threads is taken only then
      const int j0 = (tile0 + t) * kPfKeys;
      bool grow = false;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (a.cap > 0.f) {
#pragma unroll
          for (int y = 0; y < 4; ++y) s[x][y] = a.cap * tanh_f32(s[x][y] * inv_cap);
        }
        if (j0 < wlo[x] || j0 + kPfKeys > whi[x]) {
          const int rr = ty * 4 + x;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int j = j0 + tx + 16 * y;
            bool vis = j >= wlo[x] && j < whi[x];
            if (!vis && a.parent && whi[x] >= 0 && j >= P && j < hi)
              vis = (s_vis[rr][(j - P) >> 5] >> ((j - P) & 31)) & 1u;
            if (!vis) s[x][y] = -INFINITY;
          }
        }
        grow |= fmaxf(fmaxf(s[x][0], s[x][1]), fmaxf(s[x][2], s[x][3])) > m[x] + 5.5f;
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float mx = fmaxf(fmaxf(s[x][0], s[x][1]), fmaxf(s[x][2], s[x][3]));
#pragma unroll
          for (int o = 1; o < 16; o *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          if (mx > m[x]) {
            const float f = expf(m[x] - mx);  // 0 from -inf
            l[x] *= f;
#pragma unroll
            for (int u = 0; u < kU; ++u) acc[x][u][0] *= f, acc[x][u][1] *= f;
            m[x] = mx;
          }
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        // expf of a difference, not 2^(z log2 e - m): the product's rounding would cost |z| 2^-24
        const float ref = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float p = expf(s[x][y] - ref);
          l[x] += p;
          s_p[(ty * 4 + x) * S::kPStride + tx + 16 * y] = p;
        }
      }
      __syncwarp();  // a warp's rows are its own: 2 ty, 8 rows
      // ---- O += P V
      const float* pr = s_p + ty * 4 * S::kPStride;
      const float* vr = s_v + buf * kPfKeys * kD + tx * 2;
#pragma unroll 2
      for (int j = 0; j < kPfKeys; j += 4) {
        float4 pf[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) pf[x] = *reinterpret_cast<const float4*>(pr + x * S::kPStride + j);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          float2 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const float2*>(vr + (j + k) * kD + 32 * u);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            acc[x][u][0] = fmaf(pf[x].x, v[0].x, acc[x][u][0]);
            acc[x][u][1] = fmaf(pf[x].x, v[0].y, acc[x][u][1]);
            acc[x][u][0] = fmaf(pf[x].y, v[1].x, acc[x][u][0]);
            acc[x][u][1] = fmaf(pf[x].y, v[1].y, acc[x][u][1]);
            acc[x][u][0] = fmaf(pf[x].z, v[2].x, acc[x][u][0]);
            acc[x][u][1] = fmaf(pf[x].z, v[2].y, acc[x][u][1]);
            acc[x][u][0] = fmaf(pf[x].w, v[3].x, acc[x][u][0]);
            acc[x][u][1] = fmaf(pf[x].w, v[3].y, acc[x][u][1]);
          }
        }
      }
      next_q8(t, buf);
      if (!kQ8 && S::kBufs == 1 && t + 1 < t1) load_tile(t + 1, 0);
    }
    // ---- write the unit, or this CTA's part of it
    const long long c0 = kStream ? u0 / sp.per : 0, c1 = kStream ? (u1 - 1) / sp.per : 1;
    const size_t slot = kStream ? (size_t)unit_slot(blockIdx.x, sp.per, u0) : cta;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int rr = ty * 4 + x, i = (r0 + rr) / a.G, g = (r0 + rr) % a.G;
#pragma unroll
      for (int o = 1; o < 16; o *= 2) l[x] += __shfl_xor_sync(0xffffffffu, l[x], o);
      if (rr >= rows || i >= n_act) continue;
      float* to;
      float f = 1.f;
      if (c0 == c1) {
        f = 1.f / l[x];
        to = out + (((size_t)b * a.Hq + hk * a.G + g) * a.N + i) * kD;
      } else {
        to = a.ws_o + (slot * kPfRows + rr) * kD;
        if (tx == 0) __stcg(&a.ws_ml[slot * kPfRows + rr], make_float2(m[x], l[x]));
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
        __stcg(reinterpret_cast<float2*>(to + tx * 2 + 32 * u), make_float2(acc[x][u][0] * f, acc[x][u][1] * f));
    }
    if (c0 == c1) continue;
    // this CTA's rows of the merge: all of them as the last to finish, or its share of a cluster's
    int m0 = 0, m1 = rows, parts = splits;
    if constexpr (kStream) {
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        s_last = ptx::atom_add_acq_rel_gpu(&a.cnt[c0], 1u) == (unsigned)(c1 - c0);
        if (s_last) a.cnt[c0] = 0u;
        __threadfence();
      }
      __syncthreads();
      if (!s_last) continue;
      parts = (int)(c1 - c0) + 1;
    } else {
      __syncwarp();
      ptx::cluster_sync();
      m0 = rows * (int)blockIdx.x / splits;
      m1 = rows * ((int)blockIdx.x + 1) / splits;
    }
    for (int e = threadIdx.x; e < (m1 - m0) * (kD / 4); e += kPfThreads) {
      const int rr = m0 + e / (kD / 4), ch = e % (kD / 4), i = (r0 + rr) / a.G, g = (r0 + rr) % a.G;
      if (i >= n_act) continue;
      // one pass in batches of independent loads, with a running maximum
      float M = -INFINITY, L = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p0 = 0; p0 < parts; p0 += kPfMerge) {
        float2 ml[kPfMerge];
        float4 v[kPfMerge];
#pragma unroll
        for (int k = 0; k < kPfMerge; ++k) {
          const int part = min(p0 + k, parts - 1);
          const size_t from = kStream ? (size_t)unit_slot(c0 + part, sp.per, u0) : cta - blockIdx.x + part;
          ml[k] = __ldcg(&a.ws_ml[from * kPfRows + rr]);
          v[k] = __ldcg(reinterpret_cast<const float4*>(a.ws_o + (from * kPfRows + rr) * kD + ch * 4));
          if (p0 + k >= parts) ml[k].x = -INFINITY;
        }
        float Mn = M;
#pragma unroll
        for (int k = 0; k < kPfMerge; ++k) Mn = fmaxf(Mn, ml[k].x);
        if (Mn == -INFINITY) continue;
        const float f0 = expf(M - Mn);
        M = Mn;
        L *= f0;
        o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
#pragma unroll
        for (int k = 0; k < kPfMerge; ++k) {
          if (ml[k].x == -INFINITY) continue;
          const float f = expf(ml[k].x - M);
          L = fmaf(f, ml[k].y, L);
          o.x = fmaf(f, v[k].x, o.x);
          o.y = fmaf(f, v[k].y, o.y);
          o.z = fmaf(f, v[k].z, o.z);
          o.w = fmaf(f, v[k].w, o.w);
        }
      }
      const float f = 1.f / L;
      *reinterpret_cast<float4*>(out + (((size_t)b * a.Hq + hk * a.G + g) * a.N + i) * kD + ch * 4) =
          make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    }
  }
}

// ---- host side

struct PfPlan {
  int row_tiles, splits, grid;  // splits 0: persistent grid
  size_t rows, bytes;           // workspace: partial rows
};

static PfPlan pf_plan(int B, int Hq, int Hkv, int D, int N, int sms) {
  PfPlan p{};
  p.row_tiles = (Hq / Hkv * N + kPfRows - 1) / kPfRows;
  const long long units = (long long)B * Hkv * p.row_tiles;
  auto parts = [&](int n) -> int {
    const int ctas = n * (D <= 64 ? 2 : 1);
    return units * 2 <= ctas && B <= 65535 && units / B <= 65535 ? (int)min((long long)kPfMaxSplits, ctas / units) : 0;
  };
  // the workspace goes by the whole device: a share's clusters have fewer parts, and its
  // persistent grid takes two slots a CTA of what there is
  const int whole = parts(paged_device_sms());
  const size_t slots = whole ? (size_t)whole * units : (size_t)2 * kPagedMaxCtas * kPagedMaxSms;
  p.splits = parts(sms);
  p.grid = (int)min((size_t)sms * (D <= 64 ? 2 : 1), slots / 2);
  p.rows = slots * kPfRows;
  p.bytes = kPagedCntBytes + p.rows * 8 + p.rows * D * 4;
  return p;
}

template <int kD, bool kStream, bool kQ8>
static cudaError_t launch_pf_s(PagedAttn a, const PfPlan& p, cudaStream_t stream) {
  const auto fn = paged_f32_kernel<kD, kStream, kQ8>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, PfSmem<kD>::kBytes);
  if (e != cudaSuccess) return e;
  if (kStream)
    return launch_pdl(fn, dim3((unsigned)p.grid), dim3(kPfThreads), PfSmem<kD>::kBytes,
                      stream, nullptr, 0, a, 0, p.row_tiles);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  return launch_pdl(fn, dim3((unsigned)p.splits, (unsigned)(a.Hkv * p.row_tiles), (unsigned)a.B), dim3(kPfThreads),
                    PfSmem<kD>::kBytes, stream, attr, 1, a, p.splits, p.row_tiles);
}

template <int kD, bool kQ8>
static cudaError_t launch_pf(PagedAttn a, char* ws, cudaStream_t stream) {
  const PfPlan p = pf_plan(a.B, a.Hq, a.Hkv, a.D, a.N, a.sms);
  a.cnt = reinterpret_cast<unsigned*>(ws);
  a.ws_ml = reinterpret_cast<float2*>(ws + kPagedCntBytes);
  a.ws_o = reinterpret_cast<float*>(ws + kPagedCntBytes + p.rows * 8);
  return p.splits ? launch_pf_s<kD, false, kQ8>(a, p, stream) : launch_pf_s<kD, true, kQ8>(a, p, stream);
}

template <bool kQ8>
static cudaError_t launch_pf_d(const PagedAttn& a, char* ws, cudaStream_t stream) {
  switch (a.D / 32) {
    case 1:
      return launch_pf<32, kQ8>(a, ws, stream);
    case 2:
      return launch_pf<64, kQ8>(a, ws, stream);
    case 3:
      return launch_pf<96, kQ8>(a, ws, stream);
    case 4:
      return launch_pf<128, kQ8>(a, ws, stream);
    case 5:
      return launch_pf<160, kQ8>(a, ws, stream);
    case 6:
      return launch_pf<192, kQ8>(a, ws, stream);
    case 7:
      return launch_pf<224, kQ8>(a, ws, stream);
    case 8:
      return launch_pf<256, kQ8>(a, ws, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace tv
