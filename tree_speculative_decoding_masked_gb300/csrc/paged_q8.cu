// Writing, reading back and committing rows of a paged cache held in 8 bits (q8.cuh).
#include "q8.cuh"
#include "rotary.cuh"

namespace tv {

constexpr int kQaThreads = 512;  // at most
constexpr int kQaMaxRows = 128;  // rows of a tile
constexpr int kQaHeads = 2;      // heads whose loads are in flight together, and two more while they are worked on

// ---- append: new keys (normed, turned) and values into the pages, queries normed and turned
//
// A block's scale is 2^e with the least e that covers its new rows, and the scale of the committed
// rows that the block begins with; where those grow, their codes are written anew (exactly, but
// where one falls below e4m3's normal numbers).  So the scale needs the maximum over a block before
// its first code is stored: a CTA holds whole blocks of a head, a tile of rows, in registers, the
// maxima meet in shared memory, and every row is read once.  Order does not matter to a maximum, so
// results do not depend on timing.
//
// Threads: `lanes` neighbours a row, each 8 elements and their 8 pair partners (rot_to_pairs), kI rows a
// thread.  Grid: x over (sequence, tile), y over groups of hg heads of k, v and q in turn: those that wait for a
// maximum first.  64 tokens of 32 + 2 x 8 heads of 128 bf16, normed: 5.6 us, a chain of some five reads, one behind
// the other.  4 x 2048 of them, 180 MB: 44.6 us, 4.0 TB/s, bound by 16 warps an SM at 128 registers, each with some
// 250 instructions a row and head; with every number tested for being finite 48.3, queries first 49.9, without loads
// ahead of the work 59, with a branch a head 65.
template <typename T>
__device__ __forceinline__ void qa_load(const T* src, int ea, int eb, uint4 (&r)[sizeof(T)]) {
  constexpr int kHalf = sizeof(T) / 2;  // 16-byte loads of eight elements
#pragma unroll
  for (int k = 0; k < kHalf; ++k) {
    r[k] = *reinterpret_cast<const uint4*>(src + ea + k * (16 / sizeof(T)));
    r[kHalf + k] = *reinterpret_cast<const uint4*>(src + eb + k * (16 / sizeof(T)));
  }
}
template <typename T>
__device__ __forceinline__ void qa_unpack(const uint4 (&r)[sizeof(T)], float (&x)[8], float (&y)[8]) {
  if constexpr (sizeof(T) == 2) {
    rot_unpack<T, 8>(r[0], x);
    rot_unpack<T, 8>(r[1], y);
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float f[4], g[4];
      rot_unpack<T, 4>(r[k], f);
      rot_unpack<T, 4>(r[2 + k], g);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * k + i] = f[i], y[4 * k + i] = g[i];
    }
  }
}
template <typename T>
__device__ __forceinline__ float qa_number(T v) {
  if constexpr (sizeof(T) == 2)
    return bf16_to_f32(v);
  else
    return v;
}

template <typename T>
__device__ __forceinline__ void qa_store(T* dst, int ea, int eb, bool wide, const float (&x)[8], const float (&y)[8]) {
  if (!wide) {
#pragma unroll
    for (int k = 0; k < 8; ++k) dst[ea + k] = rot_pack<T, 1>({x[k]}), dst[eb + k] = rot_pack<T, 1>({y[k]});
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(dst + ea) = rot_pack<T, 8>(x);
    *reinterpret_cast<uint4*>(dst + eb) = rot_pack<T, 8>(y);
  } else {
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      *reinterpret_cast<float4*>(dst + ea + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
      *reinterpret_cast<float4*>(dst + eb + k) = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
    }
  }
}
// A row that allows single elements only: a thread's 16 in a row, each with its pair partner, read and normed again.
template <typename T>
__device__ __forceinline__ void qa_single(const RotaryArgs& a, int part, const T* src, const T* weight, long long pos,
                                          int ea, bool mine, int lanes, uint32_t peers, float inv_d, float (&x)[8],
                                          float (&y)[8]) {
  float r = 1.f;
  if (weight) {
    float ss = 0.f;
    if (mine)
      for (int k = 0; k < 16; ++k) ss = fmaf(qa_number(src[ea + k]), qa_number(src[ea + k]), ss);
    for (int o = 1; o < lanes; o *= 2) ss += __shfl_xor_sync(peers, ss, o);
    r = __frsqrt_rn(fmaf(ss, inv_d, a.eps));
  }
  auto num = [&](int d) -> float {
    const float f = qa_number(src[d]);
    return weight ? f * r * qa_number(weight[d]) : f;
  };
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    float f = 0.f;
    const int d = ea + k;
    if (mine) {
      f = num(d);
      if (part < 2 && d < a.rot) {
        const int pair = a.interleaved ? d >> 1 : d % (a.rot / 2);
        const bool upper = a.interleaved ? d & 1 : d >= a.rot / 2;
        const float other = num(a.interleaved ? d ^ 1 : upper ? d - a.rot / 2 : d + a.rot / 2);
        const float2 sc = sincos_turns((uint64_t)pos * a.freq[pair]);
        const float c = sc.y * a.amplitude, s = sc.x * a.amplitude;
        f = upper ? f * c + other * s : f * c - other * s;
      }
    }
    if (k < 8)
      x[k] = f;
    else
      y[k - 8] = f;
  }
}

// kWide: 16-byte loads, rot a multiple of 16; else single elements.
template <typename T, int kI, bool kWide, bool kInter>
__global__ void __launch_bounds__(kQaThreads) q8_append_kernel(RotaryArgs a, Q8Pages p, int tiles, int tile_rows,
                                                               int lanes, int hg) {
  constexpr int kH = kWide && kI == 1 && sizeof(T) == 2 ? kQaHeads : 1;  // as registers allow
  __shared__ int s_amax[2][kH][kQaMaxRows];
  const int b = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int kg = (a.Hkv + hg - 1) / hg;
  const int part = (int)blockIdx.y < kg ? 1 : (int)blockIdx.y < 2 * kg ? 2 : 0;
  const int h0 = part ? ((int)blockIdx.y - (part - 1) * kg) * hg : ((int)blockIdx.y - 2 * kg) * hg;
  const int h1 = part ? min(a.Hkv, h0 + hg) : min(a.Hq, h0 + hg);
  for (int k = threadIdx.x; k < 2 * kH * kQaMaxRows; k += blockDim.x) s_amax[0][0][k] = -1;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int P = a.base[b], n = a.n_rows ? a.n_rows[b] : a.N;
  if (P < 0 || n < 0 || n > a.N) {
    if (tile == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
    return;
  }
  const int bs = p.block_shift;
  const long long first = ((long long)P >> bs << bs) + (long long)tile * tile_rows;  // the tile's first cache row
  const int t_lo = (int)max(0ll, first - P), t_hi = (int)min((long long)n, first + tile_rows - P);
  if (t_lo >= t_hi) return;
  const int held = (int)max(0ll, P - first);  // committed rows that the tile's first block begins with
  const int cols = a.D / 16, col = threadIdx.x % lanes, row0 = threadIdx.x / lanes, step = blockDim.x / lanes;
  const uint32_t peers = lanes == 32 ? ~0u : ((1u << lanes) - 1u) << (threadIdx.x & 31 & -lanes);
  const bool in_row = col < cols;
  // this thread's columns: ea.. and eb..; lanes behind the row read its last ones, and bring nothing
  const int rot_cols = kWide ? a.rot / 16 : 0, c = min(col, cols - 1);
  const bool turn = kWide && part < 2 && c < rot_cols;
  int ea, eb;
  if (!kWide) {
    ea = 16 * c, eb = ea + 8;
  } else if (turn || c < rot_cols) {
    ea = 8 * c, eb = ea + a.rot / 2;
  } else {
    ea = a.rot + 8 * (c - rot_cols), eb = ea + 8 * (cols - rot_cols);
  }
  const T* weight = part < 2 ? reinterpret_cast<const T*>(a.weight[part]) : nullptr;
  const float inv_d = 1.f / a.D;
  // rows behind the tile read its last one, and bring nothing either
  const long long sh = a.sh[part];
  const T* src[kI];
#pragma unroll
  for (int i = 0; i < kI; ++i)
    src[i] = reinterpret_cast<const T*>(a.src[part]) + b * a.sb[part] +
             (long long)min(t_lo + row0 + i * step, t_hi - 1) * a.sn[part];
  // the loads of heads h and on, kH of them or one, ahead of the work on those before
  uint4 raw[kH][kI][sizeof(T)];
  auto load = [&](int h) {
    if (!kWide || h >= h1) return;
    if (h + kH <= h1) {
#pragma unroll
      for (int u = 0; u < kH; ++u)
#pragma unroll
        for (int i = 0; i < kI; ++i) qa_load<T>(src[i] + (h + u) * sh, ea, eb, raw[u][i]);
    } else {
#pragma unroll
      for (int i = 0; i < kI; ++i) qa_load<T>(src[i] + h * sh, ea, eb, raw[0][i]);
    }
  };
  load(h0);
  bool live[kI];
  long long pos[kI], page_row[kI];
  RotTurn<8> turns[kI];
#pragma unroll
  for (int i = 0; i < kI; ++i) {
    const int t = t_lo + row0 + i * step;
    live[i] = false;
    pos[i] = 0, page_row[i] = -1;
    if (t < t_hi) {
      const RotPlace at = rot_place(a, (long long)b * a.N + t, b, t, false, part > 0);
      live[i] = at.live && (part == 0 || at.page_row >= 0);
      pos[i] = at.pos, page_row[i] = at.page_row;
    }
    if (kWide && part < 2) {
      float2 wa[4], wb[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) wa[k] = wb[k] = make_float2(1.f, 1.f);
      if (weight) {
        uint4 w[sizeof(T)];
        float x[8], y[8];
        qa_load<T>(weight, ea, eb, w);
        qa_unpack<T>(w, x, y);
        rot_to_pairs<8, kInter>(x, y, wa, wb);
      }
      rot_turn_set<8, kInter>(a, pos[i], turn, c, wa, wb, turns[i]);
    }
  }
  // the page that holds the tile's first row, where that block begins with committed rows
  int held_page = -1;
  if (part && held > 0) {
    held_page = a.table[(size_t)b * a.max_pages + min(first >> a.page_shift, (long long)a.max_pages - 1)];
    if ((first >> a.page_shift) >= a.max_pages || held_page >= a.num_pages) held_page = -1;
  }
  const int in_page = (1 << a.page_shift) - 1, blocks_shift = a.page_shift - bs;
  unsigned char* cache = reinterpret_cast<unsigned char*>(part == 2 ? a.v_cache : a.k_cache);
  uint8_t* scales = part == 2 ? p.vs : p.ks;
  // the values of heads h + u, rows i, which have been loaded, to sink(u, i, x, y)
  auto values = [&](auto many, int h, auto sink) {
    constexpr int kMany = decltype(many)::value;
    if constexpr (!kWide) {
      static_assert(kMany == 1, "one head at a time");
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        float x[8], y[8];
        qa_single<T>(a, part, src[i] + h * sh, weight, pos[i], ea, live[i] && in_row, lanes, peers, inv_d, x, y);
        sink(0, i, x, y);
      }
    } else {
      if (part == 2) {
        float x[kMany][kI][8], y[kMany][kI][8];
#pragma unroll
        for (int u = 0; u < kMany; ++u)
#pragma unroll
          for (int i = 0; i < kI; ++i) qa_unpack<T>(raw[u][i], x[u][i], y[u][i]);
        load(h + kMany);
#pragma unroll
        for (int u = 0; u < kMany; ++u)
#pragma unroll
          for (int i = 0; i < kI; ++i) sink(u, i, x[u][i], y[u][i]);
        return;
      }
      float2 pa[kMany][kI][4], pb[kMany][kI][4];
      float ss[kMany][kI];
#pragma unroll
      for (int u = 0; u < kMany; ++u)
#pragma unroll
        for (int i = 0; i < kI; ++i) {
          float x[8], y[8];
          qa_unpack<T>(raw[u][i], x, y);
          rot_to_pairs<8, kInter>(x, y, pa[u][i], pb[u][i]);
          ss[u][i] = in_row ? rot_squares<8>(pa[u][i], pb[u][i]) : 0.f;
        }
      load(h + kMany);
      if (weight) {
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          if (o >= lanes) continue;
#pragma unroll
          for (int u = 0; u < kMany; ++u)
#pragma unroll
            for (int i = 0; i < kI; ++i) ss[u][i] += __shfl_xor_sync(peers, ss[u][i], o);
        }
      }
#pragma unroll
      for (int u = 0; u < kMany; ++u)
#pragma unroll
        for (int i = 0; i < kI; ++i) {
          float x[8], y[8];
          rot_turn<8>(turns[i], weight != nullptr, __frsqrt_rn(fmaf(ss[u][i], inv_d, a.eps)), turn, pa[u][i], pb[u][i]);
          rot_from_pairs<8, kInter>(pa[u][i], pb[u][i], x, y);
          sink(u, i, x, y);
        }
    }
  };
  auto queries = [&](auto many, int h) {
    const long long at = (((long long)b * a.Hq + h) * a.N + t_lo + row0) * a.D;
    values(many, h, [&](int u, int i, const float(&x)[8], const float(&y)[8]) {
      if (!kWide) __syncthreads();  // in place: the partners have been read
      if (live[i] && in_row)
        qa_store<T>(reinterpret_cast<T*>(a.q_out) + at + ((long long)u * a.N + i * step) * a.D, ea, eb, p.wide_out, x, y);
    });
  };
  auto rows = [&](auto many, int h, int buf) {
    constexpr int kMany = decltype(many)::value;
    float x[kMany][kI][8], y[kMany][kI][8];
    int old[kMany];  // the scales of the held rows
#pragma unroll
    for (int u = 0; u < kMany; ++u) {
      old[u] = 0;
      if (held_page >= 0)
        old[u] = scales[(((size_t)held_page * a.Hkv + h + u) << blocks_shift) + ((int)(first & in_page) >> bs)];
    }
    values(many, h, [&](int u, int i, const float(&v)[8], const float(&w)[8]) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[u][i][k] = v[k], y[u][i][k] = w[k];
    });
    // ---- the blocks' maxima, over what is finite
    float m[kMany][kI];
    bool odd[kMany][kI];  // something is not finite
#pragma unroll
    for (int u = 0; u < kMany; ++u)
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        float2 zero = make_float2(0.f, 0.f);  // what is finite adds 0
        m[u][i] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          zero = __ffma2_rn(make_float2(x[u][i][k], y[u][i][k]), make_float2(0.f, 0.f), zero);
          m[u][i] = fmaxf(m[u][i], fmaxf(fabsf(x[u][i][k]), fabsf(y[u][i][k])));
        }
        odd[u][i] = !(zero.x + zero.y == 0.f);
        if (odd[u][i]) {
          m[u][i] = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float f = fabsf(x[u][i][k]), g = fabsf(y[u][i][k]);
            m[u][i] = fmaxf(m[u][i], f <= 3.4028234e38f ? f : 0.f);
            m[u][i] = fmaxf(m[u][i], g <= 3.4028234e38f ? g : 0.f);
          }
        }
        if (!in_row) m[u][i] = 0.f;
      }
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      if (o >= lanes) continue;
#pragma unroll
      for (int u = 0; u < kMany; ++u)
#pragma unroll
        for (int i = 0; i < kI; ++i) m[u][i] = fmaxf(m[u][i], __shfl_xor_sync(peers, m[u][i], o));
    }
    int blk[kI];
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      blk[i] = (int)((P + (long long)(t_lo + row0 + i * step) - first) >> bs);
      if (!live[i] || col != 0) continue;
#pragma unroll
      for (int u = 0; u < kMany; ++u) atomicMax(&s_amax[buf][u][blk[i]], __float_as_int(m[u][i]));
    }
    __syncthreads();
    int first_amax[kMany];
#pragma unroll
    for (int u = 0; u < kMany; ++u) first_amax[u] = s_amax[buf][u][0];
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      if (!live[i]) continue;
#pragma unroll
      for (int u = 0; u < kMany; ++u) {
        int e = q8_exponent(__int_as_float(s_amax[buf][u][blk[i]]));
        if (blk[i] == 0 && held_page >= 0) e = max(e, old[u] - 127);
        const float f = q8_two(-e);
        const size_t row = (size_t)page_row[i] + ((size_t)(h + u) << a.page_shift);
        if (in_row) {
          unsigned char* dst = cache + row * a.D;
          float(&v)[8] = x[u][i], (&w)[8] = y[u][i];
          if (odd[u][i]) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = q8_finite(v[k]), w[k] = q8_finite(w[k]);
          }
          const float2 ff = make_float2(f, f);
          uint32_t code[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float* z = k < 2 ? v + 4 * k : w + 4 * (k - 2);
            const float2 lo = __fmul2_rn(make_float2(z[0], z[1]), ff), hi = __fmul2_rn(make_float2(z[2], z[3]), ff);
            code[k] = q8_cvt2(lo.x, lo.y) | q8_cvt2(hi.x, hi.y) << 16;
          }
          *reinterpret_cast<uint2*>(dst + ea) = make_uint2(code[0], code[1]);
          *reinterpret_cast<uint2*>(dst + eb) = make_uint2(code[2], code[3]);
        }
        // every live row of a block writes the same byte
        if (col == 0) scales[row >> bs] = (uint8_t)(e + 127);
      }
    }
    // ---- committed rows of a block whose scale has grown
#pragma unroll
    for (int u = 0; u < kMany; ++u) {
      if (held_page < 0 || first_amax[u] < 0) continue;
      const int e = q8_exponent(__int_as_float(first_amax[u]));
      if (e <= old[u] - 127) continue;
      const float ratio = q8_two(old[u] - 127 - e);
      uint4* at = reinterpret_cast<uint4*>(
          cache + ((((size_t)held_page * a.Hkv + h + u) << a.page_shift) + (size_t)(first & in_page)) * a.D);
      for (int k = threadIdx.x; k < held * cols; k += blockDim.x) {
        uint4 v = at[k];
        v.x = q8_recode(v.x, ratio), v.y = q8_recode(v.y, ratio);
        v.z = q8_recode(v.z, ratio), v.w = q8_recode(v.w, ratio);
        at[k] = v;
      }
    }
    // the other buffer is next; this one is cleared once everybody has read it, a turn later
    for (int k = threadIdx.x; k < kH * kQaMaxRows; k += blockDim.x) s_amax[buf ^ 1][0][k] = -1;
    __syncthreads();
  };

  int h = h0;
  if (part == 0) {
    for (; h + kH <= h1; h += kH) queries(std::integral_constant<int, kH>(), h);
    for (; kH > 1 && h < h1; ++h) queries(std::integral_constant<int, 1>(), h);
    return;
  }
  __syncthreads();  // s_amax is set
  int buf = 0;
  for (; h + kH <= h1; h += kH, buf ^= 1) rows(std::integral_constant<int, kH>(), h, buf);
  for (; kH > 1 && h < h1; ++h, buf ^= 1) rows(std::integral_constant<int, 1>(), h, buf);
}

template <typename T, int kI, bool kWide, bool kInter>
static cudaError_t launch_qa(const RotaryArgs& a, const Q8Pages& p, int tile_rows, int threads, int lanes,
                             cudaStream_t stream) {
  const int blk = 1 << p.block_shift;
  const long long tiles = ((long long)a.N + blk - 1 + tile_rows - 1) / tile_rows;
  if (tiles * a.B > 0x7fffffffLL) return cudaErrorInvalidValue;
  // heads share a CTA, its sines and its page lookups until the grid's warps are the 16 an SM that run at once.  As
  // many again: 4 x 2048 rows the same, one of 2048 16.6 us for 13.9, 64 single rows 6.5 for 5.5, 16 x 64 10.3 for 13.3.
  const int most = max(a.Hq, a.Hkv);
  int hg = 1;
  auto groups = [&](int g) { return (long long)(a.Hq + g - 1) / g + 2ll * ((a.Hkv + g - 1) / g); };
  while (hg < most && tiles * a.B * groups(hg) * (threads / 32) > 152 * 16) hg *= 2;
  const dim3 grid((unsigned)(tiles * a.B), (unsigned)groups(hg));
  return launch_pdl(q8_append_kernel<T, kI, kWide, kInter>, grid, dim3(threads), 0, stream, nullptr, 0, a, p,
                    (int)tiles, tile_rows, lanes, hg);
}

template <typename T>
static cudaError_t launch_qa_t(const RotaryArgs& a, Q8Pages p, cudaStream_t stream) {
  bool wide = a.rot % 16 == 0;
  constexpr int vec = 16 / sizeof(T);
  for (int i = 0; i < 3; ++i)
    if (a.src[i])
      wide = wide && reinterpret_cast<uintptr_t>(a.src[i]) % 16 == 0 && a.sb[i] % vec == 0 && a.sh[i] % vec == 0 &&
             a.sn[i] % vec == 0;
  for (const void* w : a.weight) wide = wide && reinterpret_cast<uintptr_t>(w) % 16 == 0;
  p.wide_out = reinterpret_cast<uintptr_t>(a.q_out) % 16 == 0;
  int lanes = 2;  // D / 16 columns, up to the next power of two
  while (lanes * 16 < a.D) lanes *= 2;
  // whole blocks, a row a thread where 512 threads allow it; calls of few rows need no more threads than those
  const int tile_rows = max(1 << p.block_shift, 256 / lanes), all = tile_rows * lanes;
  const int threads = (int)min((long long)min(all, kQaThreads), ((long long)a.N * lanes + 31) / 32 * 32);
  if (all > kQaThreads && (long long)a.N * lanes > kQaThreads)
    return !wide           ? launch_qa<T, 2, false, false>(a, p, tile_rows, threads, lanes, stream)
           : a.interleaved ? launch_qa<T, 2, true, true>(a, p, tile_rows, threads, lanes, stream)
                           : launch_qa<T, 2, true, false>(a, p, tile_rows, threads, lanes, stream);
  return !wide           ? launch_qa<T, 1, false, false>(a, p, tile_rows, threads, lanes, stream)
         : a.interleaved ? launch_qa<T, 1, true, true>(a, p, tile_rows, threads, lanes, stream)
                         : launch_qa<T, 1, true, false>(a, p, tile_rows, threads, lanes, stream);
}

cudaError_t launch_q8_append(const RotaryArgs& a, const Q8Pages& p, tv_dtype dtype, cudaStream_t stream) {
  return dtype == TV_BF16 ? launch_qa_t<uint16_t>(a, p, stream) : launch_qa_t<float>(a, p, stream);
}

// ---- read back: rows first_b + r < length_b of the cache to row r of contiguous [B][Hkv][rows][D]
//
// One pass over memory, 8 codes a thread and row: a row's codes are read in order and its numbers written
// in order.  Exact in bf16: a code has four significant bits.  8 sequences of 8192 to 16384 rows, 8 heads of 128, 500
// MB: 89 us, 5.6 TB/s, memory; one of 2048: 4.3 us.
constexpr int kQrThreads = 256;
constexpr int kQrRows = 4;  // rows a thread has in flight

template <typename T>
__global__ void __launch_bounds__(kQrThreads) q8_read_kernel(Q8Read a) {
  const int cols = a.D / 8, col = threadIdx.x % cols, step = kQrThreads / cols, row0 = threadIdx.x / cols;
  const int h = blockIdx.y, b = blockIdx.z;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int first = a.first ? a.first[b] : 0, length = a.length[b];
  if (first < 0 || length < 0) {
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
    return;
  }
  if (row0 >= step) return;
  const long long r0 = (long long)blockIdx.x * step * kQrRows + row0;
  const long long n = min((long long)a.rows, (long long)length - first);
  uint2 kc[kQrRows], vc[kQrRows];
  unsigned ks[kQrRows], vs[kQrRows];
  bool have[kQrRows];
#pragma unroll
  for (int u = 0; u < kQrRows; ++u) {
    const long long r = r0 + (long long)u * step, j = first + r, pg = j >> a.page_shift;
    have[u] = false;
    if (r < n) {
      const int page = pg < a.max_pages ? a.table[(size_t)b * a.max_pages + pg] : -1;
      have[u] = page >= 0 && page < a.num_pages;
      if (!have[u]) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
      if (have[u]) {
        const size_t row = (((size_t)page * a.Hkv + h) << a.page_shift) + (size_t)(j & ((1 << a.page_shift) - 1));
        kc[u] = *reinterpret_cast<const uint2*>(a.k + row * a.D + col * 8);
        vc[u] = *reinterpret_cast<const uint2*>(a.v + row * a.D + col * 8);
        ks[u] = a.ks[row >> a.block_shift];
        vs[u] = a.vs[row >> a.block_shift];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kQrRows; ++u) {
    if (!have[u]) continue;
    const size_t at = (((size_t)b * a.Hkv + h) * a.rows + (size_t)(r0 + (long long)u * step)) * a.D + col * 8;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint2 c = kv ? vc[u] : kc[u];
      const float s = q8_scale(kv ? vs[u] : ks[u]);
      const float4 x = q8_numbers(c.x, s), y = q8_numbers(c.y, s);
      T* dst = reinterpret_cast<T*>(kv ? a.v_out : a.k_out) + at;
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(ptx::cvt_bf16x2(x.x, x.y), ptx::cvt_bf16x2(x.z, x.w),
                                                    ptx::cvt_bf16x2(y.x, y.y), ptx::cvt_bf16x2(y.z, y.w));
      } else {
        *reinterpret_cast<float4*>(dst) = x;
        *reinterpret_cast<float4*>(dst + 4) = y;
      }
    }
  }
}

cudaError_t launch_q8_read(const Q8Read& a, tv_dtype dtype, cudaStream_t stream) {
  const int per = kQrThreads / (a.D / 8) * kQrRows;
  const dim3 grid((unsigned)((a.rows + per - 1) / per), (unsigned)a.Hkv, (unsigned)a.B);
  return launch_pdl(dtype == TV_BF16 ? q8_read_kernel<uint16_t> : q8_read_kernel<float>, grid, dim3(kQrThreads), 0,
                    stream, nullptr, 0, a);
}

// ---- commit: row P + a_k to row P + k, k = 1..L
//
// A block that receives rows takes the largest scale of its own and of the blocks that the rows come from;
// rows that change their scale, the live ones before the path in the first block among them, are coded
// anew.  One CTA a (sequence, KV head, K or V), tile after tile of 64 destination rows in whole blocks: a
// tile's sources, and their scales, are all read before anything of it is written, and since a_k >= k
// and the a_k increase, no later tile reads a row or a scale that an earlier one wrote.  64 paths of 8 to 16 rows, 8
// heads of 128: 5.7 us, one of 5 2.8: dependent reads (lengths, path, pages, rows and scales) and four barriers.
constexpr int kQcThreads = 256;
constexpr int kQcRows = 64;

__global__ void __launch_bounds__(kQcThreads)
    q8_commit_kernel(unsigned char* k_cache, unsigned char* v_cache, Q8Pages p, const int32_t* table,
                     const int32_t* prefix_len, const int32_t* accepted, const int32_t* accept_len, int32_t* new_len,
                     int Hkv, int N, int num_pages, int page_shift, int max_pages, int D, int32_t* dev_status) {
  __shared__ int s_scale[kQcRows];  // of the tile's blocks, when it is done
  const int b = blockIdx.y, h = blockIdx.x >> 1;
  unsigned char* cache = (blockIdx.x & 1) ? v_cache : k_cache;
  uint8_t* scales = (blockIdx.x & 1) ? p.vs : p.ks;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int len = accept_len[b], P = prefix_len[b], bs = p.block_shift;
  const int32_t* acc = accepted + (size_t)b * N;
  const int32_t* tab = table + (size_t)b * max_pages;
  if (len < 0 || len >= N || P < 0) {
    if (threadIdx.x == 0) set_dev_status(dev_status, P < 0 ? TV_DEV_BAD_PAGE : TV_DEV_BAD_TREE);
    return;
  }
  if (new_len && blockIdx.x == 0 && threadIdx.x == 0) new_len[b] = P + len + 1;
  const int chunks = D / 16;
  auto place = [&](long long r) -> long long {  // cache row r's row in the pool, or -1
    const long long pg = r >> page_shift;
    const int page = pg < max_pages ? tab[pg] : -1;
    if (page < 0 || page >= num_pages) {
      set_dev_status(dev_status, TV_DEV_BAD_PAGE);
      return -1;
    }
    return (((long long)page * Hkv + h) << page_shift) + (r & ((1 << page_shift) - 1));
  };
  const long long begin = (long long)P + 1, end = begin + len;
  for (long long first = begin >> bs << bs; first < end && len > 0; first += kQcRows) {
    const long long lo = max(first, begin), hi = min(first + kQcRows, end);
    const int rows = (int)(hi - lo), items = rows * chunks;
    for (int k = threadIdx.x; k < kQcRows; k += kQcThreads) s_scale[k] = -1;
    __syncthreads();
    uint4 val[kQcRows * 16 / kQcThreads];
    long long dst[kQcRows * 16 / kQcThreads];
    int from[kQcRows * 16 / kQcThreads];  // the scale that the value has; bit 8: it moves
#pragma unroll
    for (int u = 0; u < kQcRows * 16 / kQcThreads; ++u) {
      const int e = u * kQcThreads + threadIdx.x;
      dst[u] = -1;
      if (e >= items) continue;
      const int ch = e % chunks, k = (int)(lo - begin) + e / chunks + 1;
      const int at = acc[k - 1], prev = k > 1 ? acc[k - 2] : 0;
      if (at <= prev || at < k || at >= N) {  // a root path has increasing node ids
        set_dev_status(dev_status, TV_DEV_BAD_TREE);
        continue;
      }
      const long long src = place((long long)P + at), to = place((long long)P + k);
      if (src < 0 || to < 0) continue;
      val[u] = *reinterpret_cast<const uint4*>(cache + (size_t)src * D + ch * 16);
      dst[u] = to;
      const int s = scales[src >> bs];
      from[u] = s | (at != k ? 256 : 0);
      if (ch == 0) atomicMax(&s_scale[(int)((P + (long long)k - first) >> bs)], max(s, (int)scales[to >> bs]));
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kQcRows * 16 / kQcThreads; ++u) {
      if (dst[u] < 0) continue;
      const int e = u * kQcThreads + threadIdx.x, ch = e % chunks;
      const int to = s_scale[(int)((lo - first + e / chunks) >> bs)], s = from[u] & 255;
      if (to > s) {
        const float ratio = q8_two(s - to);
        val[u].x = q8_recode(val[u].x, ratio), val[u].y = q8_recode(val[u].y, ratio);
        val[u].z = q8_recode(val[u].z, ratio), val[u].w = q8_recode(val[u].w, ratio);
      }
      if (to > s || from[u] & 256) *reinterpret_cast<uint4*>(cache + (size_t)dst[u] * D + ch * 16) = val[u];
    }
    // live rows before the path, and the blocks' scales
    const int held = (int)(lo - first), to0 = s_scale[0];
    if (held > 0 && to0 >= 0) {
      const long long row = place(first);
      const int s = row < 0 ? 255 : scales[row >> bs];
      if (to0 > s) {
        const float ratio = q8_two(s - to0);
        uint4* at = reinterpret_cast<uint4*>(cache + (size_t)row * D);
        for (int k = threadIdx.x; k < held * chunks; k += kQcThreads) {
          uint4 v = at[k];
          v.x = q8_recode(v.x, ratio), v.y = q8_recode(v.y, ratio);
          v.z = q8_recode(v.z, ratio), v.w = q8_recode(v.w, ratio);
          at[k] = v;
        }
      }
    }
    __syncthreads();  // the first block's scale has been read
    for (int k = threadIdx.x; k < (kQcRows >> bs); k += kQcThreads)
      if (s_scale[k] >= 0) {
        const long long row = place(max(first + ((long long)k << bs), lo));
        if (row >= 0) scales[row >> bs] = (uint8_t)s_scale[k];
      }
    __syncthreads();
  }
}

cudaError_t launch_q8_commit(void* k, void* v, const Q8Pages& p, const int32_t* table, const int32_t* prefix_len,
                             const int32_t* accepted, const int32_t* accept_len, int32_t* new_len, int B, int Hkv,
                             int D, int N, int num_pages, int page_shift, int max_pages, int32_t* dev_status,
                             cudaStream_t stream) {
  return launch_pdl(q8_commit_kernel, dim3((unsigned)(2 * Hkv), (unsigned)B), dim3(kQcThreads), 0, stream, nullptr, 0,
                    reinterpret_cast<unsigned char*>(k), reinterpret_cast<unsigned char*>(v), p, table, prefix_len,
                    accepted, accept_len, new_len, Hkv, N, num_pages, page_shift, max_pages, D, dev_status);
}

}  // namespace tv
