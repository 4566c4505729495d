// Writing, reading back and committing rows of a paged cache held in 8 bits (q8.cuh).
#include "q8.cuh"
#include "rotary.cuh"

namespace tv {

constexpr int kQaThreads = 256;
constexpr int kQaMaxRows = 128;  // rows of a tile

// ---- append: new keys (normed, turned) and values into the pages, queries normed and turned
//
// A block's scale is 2^e with the least e that covers its new rows, and the scale of the committed
// rows that the block begins with; where those grow, their codes are written anew (exactly, but
// where one falls below e4m3's normal numbers).  So the scale needs the maximum over a block before
// its first code is stored: a CTA holds whole blocks of one head, a tile of up to 64 rows (128 of 32
// elements), in registers, the maxima meet in shared memory, and every row is read once.  Order does
// not matter to a maximum, so results do not depend on timing.
//
// Threads: `lanes` neighbours a row, each 8 elements and their 8 pair partners (as in rotary_kernel),
// kI rows a thread.  Grid: x over (sequence, tile), y over groups of hg heads of q, k and v in turn.
template <typename T, bool kWide>
__device__ __forceinline__ void qa_load(const T* src, int ea, int eb, uint4 (&r)[sizeof(T)]) {
  if constexpr (kWide) {
    constexpr int kHalf = sizeof(T) / 2;  // 16-byte loads of eight elements
#pragma unroll
    for (int k = 0; k < kHalf; ++k) {
      r[k] = *reinterpret_cast<const uint4*>(src + ea + k * (16 / sizeof(T)));
      r[kHalf + k] = *reinterpret_cast<const uint4*>(src + eb + k * (16 / sizeof(T)));
    }
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

// kWide: 16-byte loads, rot a multiple of 16.  Else single elements, a thread's 16 in a row, each with its
// pair partner (read and normed again).
template <typename T, int kI, bool kWide>
__global__ void __launch_bounds__(kQaThreads) q8_append_kernel(RotaryArgs a, Q8Pages p, int tiles, int tile_rows,
                                                               int lanes, int hg) {
  __shared__ int s_amax[2][kQaMaxRows];
  const int b = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int qg = (a.Hq + hg - 1) / hg, kg = (a.Hkv + hg - 1) / hg;
  const int part = (int)blockIdx.y < qg ? 0 : (int)blockIdx.y < qg + kg ? 1 : 2;
  const int h0 = ((int)blockIdx.y - (part == 0 ? 0 : part == 1 ? qg : qg + kg)) * hg;
  const int h1 = min(part ? a.Hkv : a.Hq, h0 + hg);
  for (int k = threadIdx.x; k < 2 * kQaMaxRows; k += blockDim.x) s_amax[0][k] = -1;
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
  // this thread's columns: ea.. and eb..
  const int rot_cols = kWide ? a.rot / 16 : 0;
  const bool turn = kWide && part < 2 && col < rot_cols;
  int ea, eb;
  if (!kWide) {
    ea = 16 * col, eb = ea + 8;
  } else if (col < rot_cols) {
    ea = 8 * col, eb = ea + a.rot / 2;
  } else {
    ea = a.rot + 8 * (col - rot_cols), eb = ea + 8 * (cols - rot_cols);
  }
  bool live[kI];
  long long pos[kI], page_row[kI];
  float cs[kI][8], sn[kI][8];
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
    if (turn && live[i]) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int pair = a.interleaved ? (u < 4 ? 0 : a.rot / 4 - 4) + 4 * col + u : 8 * col + u;
        const float2 sc = sincos_turns((uint64_t)pos[i] * a.freq[pair]);
        sn[i][u] = sc.x * a.amplitude;
        cs[i][u] = sc.y * a.amplitude;
      }
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

  __syncthreads();  // s_amax is set
  for (int h = h0, buf = 0; h < h1; ++h, buf ^= 1) {
    float x[kI][8], y[kI][8];
    uint4 raw[kI][sizeof(T)];
#pragma unroll
    for (int i = 0; i < kI; ++i)
      if (kWide && live[i] && in_row)
        qa_load<T, kWide>(reinterpret_cast<const T*>(a.src[part]) + b * a.sb[part] + h * a.sh[part] +
                              (long long)(t_lo + row0 + i * step) * a.sn[part],
                          ea, eb, raw[i]);
    int old = 0;  // the scale of the held rows
    const size_t held_scale =
        held_page < 0 ? 0 : (((size_t)held_page * a.Hkv + h) << blocks_shift) + ((int)(first & in_page) >> bs);
    if (held_page >= 0) old = scales[held_scale];
#pragma unroll
    for (int i = 0; i < kI; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[i][k] = y[i][k] = 0.f;
      if (kWide) {
        if (live[i] && in_row) qa_unpack<T>(raw[i], x[i], y[i]);
        if (part < 2 && a.weight[part]) {
          // sums of squares meet over the row's lanes, live or not alike
          float ss = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) ss = fmaf(x[i][k], x[i][k], fmaf(y[i][k], y[i][k], ss));
          for (int o = 1; o < lanes; o *= 2) ss += __shfl_xor_sync(peers, ss, o);
          const float r = 1.f / sqrtf(ss / a.D + a.eps);
          if (in_row) {
            const T* weight = reinterpret_cast<const T*>(a.weight[part]);
            uint4 wr[sizeof(T)];
            float wx[8], wy[8];
            qa_load<T, kWide>(weight, ea, eb, wr);
            qa_unpack<T>(wr, wx, wy);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[i][k] = x[i][k] * r * wx[k], y[i][k] = y[i][k] * r * wy[k];
          }
        }
        if (turn) {
          if (a.interleaved) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float e0 = x[i][2 * k], o0 = x[i][2 * k + 1], e1 = y[i][2 * k], o1 = y[i][2 * k + 1];
              x[i][2 * k] = e0 * cs[i][k] - o0 * sn[i][k];
              x[i][2 * k + 1] = o0 * cs[i][k] + e0 * sn[i][k];
              y[i][2 * k] = e1 * cs[i][4 + k] - o1 * sn[i][4 + k];
              y[i][2 * k + 1] = o1 * cs[i][4 + k] + e1 * sn[i][4 + k];
            }
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float e = x[i][k], o = y[i][k];
              x[i][k] = e * cs[i][k] - o * sn[i][k];
              y[i][k] = o * cs[i][k] + e * sn[i][k];
            }
          }
        }
      } else {
        const T* src = reinterpret_cast<const T*>(a.src[part]) + b * a.sb[part] + h * a.sh[part] +
                       (long long)(t_lo + row0 + i * step) * a.sn[part];
        const bool mine = live[i] && in_row;
        float r = 1.f;
        const T* weight = part < 2 ? reinterpret_cast<const T*>(a.weight[part]) : nullptr;
        if (weight) {
          float ss = 0.f;
          if (mine)
            for (int k = 0; k < 16; ++k) ss = fmaf(qa_number(src[ea + k]), qa_number(src[ea + k]), ss);
          for (int o = 1; o < lanes; o *= 2) ss += __shfl_xor_sync(peers, ss, o);
          r = 1.f / sqrtf(ss / a.D + a.eps);
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
              const float2 sc = sincos_turns((uint64_t)pos[i] * a.freq[pair]);
              const float c = sc.y * a.amplitude, s = sc.x * a.amplitude;
              f = upper ? f * c + other * s : f * c - other * s;
            }
          }
          if (k < 8)
            x[i][k] = f;
          else
            y[i][k - 8] = f;
        }
      }
    }
    if (part == 0) {
      if (!kWide) __syncthreads();  // in place: the partners have been read
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        if (!live[i] || !in_row) continue;
        T* dst = reinterpret_cast<T*>(a.q_out) +
                 (((long long)b * a.Hq + h) * a.N + t_lo + row0 + i * step) * a.D;
        if (p.wide_out) {
          if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(dst + ea) = rot_pack<T, 8>(x[i]);
            *reinterpret_cast<uint4*>(dst + eb) = rot_pack<T, 8>(y[i]);
          } else {
#pragma unroll
            for (int k = 0; k < 8; k += 4) {
              *reinterpret_cast<float4*>(dst + ea + k) = make_float4(x[i][k], x[i][k + 1], x[i][k + 2], x[i][k + 3]);
              *reinterpret_cast<float4*>(dst + eb + k) = make_float4(y[i][k], y[i][k + 1], y[i][k + 2], y[i][k + 3]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if constexpr (sizeof(T) == 2) {
              dst[ea + k] = (T)(ptx::cvt_bf16x2(x[i][k], 0.f) & 0xffffu);
              dst[eb + k] = (T)(ptx::cvt_bf16x2(y[i][k], 0.f) & 0xffffu);
            } else {
              dst[ea + k] = x[i][k];
              dst[eb + k] = y[i][k];
            }
          }
        }
      }
      continue;
    }
    // ---- the blocks' maxima, over what is finite
    int blk[kI];
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float u = fabsf(x[i][k]), w = fabsf(y[i][k]);
        m = fmaxf(m, u <= 3.4028234e38f ? u : 0.f);
        m = fmaxf(m, w <= 3.4028234e38f ? w : 0.f);
      }
      for (int o = 1; o < lanes; o *= 2) m = fmaxf(m, __shfl_xor_sync(peers, m, o));
      blk[i] = (int)((P + (long long)(t_lo + row0 + i * step) - first) >> bs);
      if (live[i] && col == 0) atomicMax(&s_amax[buf][blk[i]], __float_as_int(m));
    }
    __syncthreads();
    const int first_amax = s_amax[buf][0];
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      if (!live[i]) continue;
      int e = q8_exponent(__int_as_float(s_amax[buf][blk[i]]));
      if (blk[i] == 0 && held_page >= 0) e = max(e, old - 127);
      const float f = q8_two(-e);
      const size_t row = (size_t)page_row[i] + ((size_t)h << a.page_shift);
      if (in_row) {
        unsigned char* dst = cache + row * a.D;
        uint2 lo, hi;
        lo.x = q8_code4(x[i][0] * f, x[i][1] * f, x[i][2] * f, x[i][3] * f);
        lo.y = q8_code4(x[i][4] * f, x[i][5] * f, x[i][6] * f, x[i][7] * f);
        hi.x = q8_code4(y[i][0] * f, y[i][1] * f, y[i][2] * f, y[i][3] * f);
        hi.y = q8_code4(y[i][4] * f, y[i][5] * f, y[i][6] * f, y[i][7] * f);
        *reinterpret_cast<uint2*>(dst + ea) = lo;
        *reinterpret_cast<uint2*>(dst + eb) = hi;
      }
      // every live row of a block writes the same byte
      if (col == 0) scales[row >> bs] = (uint8_t)(e + 127);
    }
    // ---- committed rows of a block whose scale has grown
    if (held_page >= 0 && first_amax >= 0) {
      const int e = q8_exponent(__int_as_float(first_amax));
      if (e > old - 127) {
        const float ratio = q8_two(old - 127 - e);
        uint4* rows = reinterpret_cast<uint4*>(
            cache + ((((size_t)held_page * a.Hkv + h) << a.page_shift) + (size_t)(first & in_page)) * a.D);
        for (int k = threadIdx.x; k < held * cols; k += blockDim.x) {
          uint4 v = rows[k];
          v.x = q8_recode(v.x, ratio), v.y = q8_recode(v.y, ratio);
          v.z = q8_recode(v.z, ratio), v.w = q8_recode(v.w, ratio);
          rows[k] = v;
        }
      }
    }
    // the other buffer is next; this one is cleared once everybody has read it, a head later
    for (int k = threadIdx.x; k < kQaMaxRows; k += blockDim.x) s_amax[buf ^ 1][k] = -1;
    __syncthreads();
  }
}

template <typename T, int kI, bool kWide>
static cudaError_t launch_qa(const RotaryArgs& a, const Q8Pages& p, int threads, int lanes, cudaStream_t stream) {
  const int blk = 1 << p.block_shift;
  const int tile_rows = max(64, 256 / lanes);
  const long long tiles = ((long long)a.N + blk - 1 + tile_rows - 1) / tile_rows;
  if (tiles * a.B > 0x7fffffffLL) return cudaErrorInvalidValue;
  // heads share a CTA, its sines and its page lookups once the grid has a few CTAs an SM without that
  const int most = max(a.Hq, a.Hkv);
  int hg = 1;
  auto groups = [&](int g) { return (long long)(a.Hq + g - 1) / g + 2ll * ((a.Hkv + g - 1) / g); };
  while (hg < most && tiles * a.B * groups(hg) > 152 * 16) hg *= 2;
  const dim3 grid((unsigned)(tiles * a.B), (unsigned)groups(hg));
  return launch_pdl(q8_append_kernel<T, kI, kWide>, grid, dim3(threads), 0, stream, nullptr, 0, a, p, (int)tiles,
                    tile_rows, lanes, hg);
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
  // a tile's rows, 64 or more, over 256 threads; calls of few rows need no more than those
  if ((long long)a.N * lanes <= kQaThreads || lanes <= 4) {
    const int threads = min(kQaThreads, (a.N * lanes + 31) / 32 * 32);
    return wide ? launch_qa<T, 1, true>(a, p, threads, lanes, stream)
                : launch_qa<T, 1, false>(a, p, threads, lanes, stream);
  }
  if (lanes == 8)
    return wide ? launch_qa<T, 2, true>(a, p, kQaThreads, lanes, stream)
                : launch_qa<T, 2, false>(a, p, kQaThreads, lanes, stream);
  return wide ? launch_qa<T, 4, true>(a, p, kQaThreads, lanes, stream)
              : launch_qa<T, 4, false>(a, p, kQaThreads, lanes, stream);
}

cudaError_t launch_q8_append(const RotaryArgs& a, const Q8Pages& p, tv_dtype dtype, cudaStream_t stream) {
  return dtype == TV_BF16 ? launch_qa_t<uint16_t>(a, p, stream) : launch_qa_t<float>(a, p, stream);
}

// ---- read back: rows first_b + r < length_b of the cache to row r of contiguous [B][Hkv][rows][D]
//
// One pass over memory, 8 codes a thread and row: a row's codes are read in order and its numbers written
// in order.  Exact in bf16: a code has four significant bits.
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
// and the a_k increase, no later tile reads a row or a scale that an earlier one wrote.
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
