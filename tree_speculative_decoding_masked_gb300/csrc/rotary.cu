// Rotary positions, and the append of new keys and values to a paged cache with the
// rotation on the way.
//
// A head's first R of D elements form R / 2 pairs; pair i of a row at position p turns by
// the angle p f_i:  (x, y) -> A (x cos - y sin, y cos + x sin).  Pairs are (i, i + R/2) ("half")
// or (2i, 2i + 1) ("interleaved"); A is the amplitude of the frequency scaling (1 for most).
// The frequencies are held as f_i / 2 pi in units of 2^-64 turns, so the angle's fraction of a
// turn is the low 64 bits of the integer product p f: exact at any position, where a
// 32-bit product would be off by p 2^-24 radians.
//
// The work is one pass over memory.  A thread owns 16 bytes and their pair partners of one
// token, takes the sines and cosines of its pairs once, and turns those columns of all the
// heads of its group; the groups are sized so that small batches still fill the device.
#include <math.h>

#include "paged.cuh"

namespace tv {

constexpr int kRotThreads = 256;

// kVec contiguous elements as floats
template <typename T, int kVec>
__device__ __forceinline__ void rot_load(const T* p, float (&f)[kVec]) {
  if constexpr (kVec == 1) {
    if constexpr (sizeof(T) == 2)
      f[0] = bf16_to_f32(*p);
    else
      f[0] = *p;
  } else if constexpr (sizeof(T) == 2) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  }
}
template <typename T, int kVec>
__device__ __forceinline__ void rot_store(T* p, const float (&f)[kVec]) {
  if constexpr (kVec == 1) {
    if constexpr (sizeof(T) == 2)
      *p = (T)(ptx::cvt_bf16x2(f[0], 0.f) & 0xffffu);
    else
      *p = f[0];
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(ptx::cvt_bf16x2(f[0], f[1]), ptx::cvt_bf16x2(f[2], f[3]),
                                              ptx::cvt_bf16x2(f[4], f[5]), ptx::cvt_bf16x2(f[6], f[7]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
}
// kVec contiguous elements unchanged (a NaN's bits survive)
template <typename T, int kVec>
__device__ __forceinline__ void rot_copy(T* dst, const T* src) {
  if constexpr (kVec == 1)
    *dst = *src;
  else
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
}

// Grid: x over (token, column) pairs, y over groups of `hg` of the Hq + 2 Hkv heads.  A column
// is kVec pairs (rotated part) or up to 2 kVec elements behind it.
template <typename T, int kVec>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(RotaryArgs a, int cols, int rot_cols, int hg) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const long long id = (long long)blockIdx.x * kRotThreads + threadIdx.x;
  const long long token = id / cols;
  if (token >= (long long)a.B * a.N) return;
  const int col = (int)(id - token * cols);
  const int b = (int)(token / a.N), t = (int)(token - (long long)b * a.N);
  const int off = a.pos ? a.pos[token] : t;
  if (off < 0) return;  // padding
  const int base = a.base ? a.base[b] : 0;
  if (a.n_rows && t >= a.n_rows[b]) return;
  const long long p = (long long)base + off;
  const int heads = a.Hq + 2 * a.Hkv;
  const int h0 = blockIdx.y * hg, h1 = min(heads, h0 + hg);
  // where this token's row goes in a page
  long long page_row = -1;
  if (h1 > a.Hq) {
    const long long r = (long long)base + t;
    const long long pg = r >> a.page_shift;
    const int page = base >= 0 && pg < a.max_pages ? a.table[(size_t)b * a.max_pages + pg] : -1;
    if (page >= 0 && page < a.num_pages)
      page_row = ((long long)page * a.Hkv << a.page_shift) + (r & ((1 << a.page_shift) - 1));
    else
      set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
  }
  if (p < 0) return;  // a negative base
  // this thread's elements: ea.. and eb.. (eb == D: none)
  const bool turn = col < rot_cols;
  int ea, eb;
  if (turn) {
    ea = a.interleaved ? 2 * kVec * col : kVec * col;
    eb = a.interleaved ? ea + kVec : ea + a.rot / 2;
  } else {
    ea = a.rot + 2 * kVec * (col - rot_cols);
    eb = min(a.D, ea + kVec);
  }
  float cs[kVec], sn[kVec];
  if (turn && h0 < a.Hq + a.Hkv) {
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      const uint64_t turns = (uint64_t)p * a.freq[kVec * col + u];
      // a signed half turn in 2^-31 steps: within 2^-31 pi of the angle
      const float half = (float)(int)(turns >> 32) * 0x1p-31f;
      sincospif(half, &sn[u], &cs[u]);
      sn[u] *= a.amplitude;
      cs[u] *= a.amplitude;
    }
  }
  for (int h = h0; h < h1; ++h) {
    const int part = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2;
    const int hh = part == 0 ? h : part == 1 ? h - a.Hq : h - a.Hq - a.Hkv;
    const T* src = reinterpret_cast<const T*>(a.src[part]) + b * a.sb[part] + hh * a.sh[part] + t * a.sn[part];
    T* dst;
    if (part == 0) {
      dst = reinterpret_cast<T*>(a.q_out) + (((long long)b * a.Hq + hh) * a.N + t) * a.D;
    } else {
      if (page_row < 0) continue;
      dst = reinterpret_cast<T*>(part == 1 ? a.k_cache : a.v_cache) +
            (page_row + ((long long)hh << a.page_shift)) * a.D;
    }
    if (part == 2 || !turn) {
      rot_copy<T, kVec>(dst + ea, src + ea);
      if (eb < a.D) rot_copy<T, kVec>(dst + eb, src + eb);
      continue;
    }
    float x[kVec], y[kVec];
    rot_load<T, kVec>(src + ea, x);
    rot_load<T, kVec>(src + eb, y);
    if (a.interleaved && kVec > 1) {
      // x, y hold 2 kVec contiguous elements: pair u is elements 2u, 2u + 1
#pragma unroll
      for (int u = 0; u < kVec / 2; ++u) {
        const float e0 = x[2 * u], o0 = x[2 * u + 1], e1 = y[2 * u], o1 = y[2 * u + 1];
        x[2 * u] = e0 * cs[u] - o0 * sn[u];
        x[2 * u + 1] = o0 * cs[u] + e0 * sn[u];
        y[2 * u] = e1 * cs[kVec / 2 + u] - o1 * sn[kVec / 2 + u];
        y[2 * u + 1] = o1 * cs[kVec / 2 + u] + e1 * sn[kVec / 2 + u];
      }
    } else {
#pragma unroll
      for (int u = 0; u < kVec; ++u) {
        const float e = x[u], o = y[u];
        x[u] = e * cs[u] - o * sn[u];
        y[u] = o * cs[u] + e * sn[u];
      }
    }
    rot_store<T, kVec>(dst + ea, x);
    rot_store<T, kVec>(dst + eb, y);
  }
}

template <typename T, int kVec>
static cudaError_t launch_rot(const RotaryArgs& a, cudaStream_t stream) {
  const int rot_cols = a.rot / (2 * kVec);
  const int rest = a.D - a.rot;
  const int cols = rot_cols + (rest + 2 * kVec - 1) / (2 * kVec);
  const int heads = a.Hq + 2 * a.Hkv;
  const long long threads = (long long)a.B * a.N * cols;
  const long long blocks = (threads + kRotThreads - 1) / kRotThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  int hg = 1;
  while (hg < heads && blocks * ((heads + hg - 1) / hg) > 152 * 8) hg *= 2;
  const dim3 grid((unsigned)blocks, (unsigned)((heads + hg - 1) / hg));
  return launch_pdl(rotary_kernel<T, kVec>, grid, dim3(kRotThreads), 0, stream, nullptr, 0, a, cols, rot_cols, hg);
}

cudaError_t launch_rotary(const RotaryArgs& a, tv_dtype dtype, cudaStream_t stream) {
  const int vec = dtype == TV_BF16 ? 8 : 4;
  // 16-byte columns where every row, pair half and stride allows them, else one element a
  // thread and pair half
  bool wide = a.D % vec == 0 && a.rot % (2 * vec) == 0;
  for (int i = 0; i < 3; ++i)
    if (a.src[i])
      wide = wide && reinterpret_cast<uintptr_t>(a.src[i]) % 16 == 0 && a.sb[i] % vec == 0 && a.sh[i] % vec == 0 &&
             a.sn[i] % vec == 0;
  for (const void* p : {(const void*)a.q_out, (const void*)a.k_cache, (const void*)a.v_cache})
    wide = wide && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  if (dtype == TV_BF16) return wide ? launch_rot<uint16_t, 8>(a, stream) : launch_rot<uint16_t, 1>(a, stream);
  return wide ? launch_rot<float, 4>(a, stream) : launch_rot<float, 1>(a, stream);
}

// Frequencies in 2^-64 turns a position.  With r_i = base^(-2i/R) radians:
//   none   r_i
//   linear r_i / s                                    params {s}
//   base   (base s^(R/(R-2)))^(-2i/R)                 params {s}
//   banded r_i (m + (1 - m) / s), m = clamp((L r_i / 2 pi - lo) / (hi - lo), 0, 1):
//          pairs that turn more than hi times in L positions keep their pace, those that
//          turn less than lo times are slowed by s    params {s, lo, hi, L}
//   yarn   r_i (k + (1 - k) / s), k falling from 1 to 0 between the pairs that turn `fast`
//          and `slow` times in L positions; amplitude 0.1 ln s + 1 (Peng et al., "YaRN:
//          efficient context window extension of large language models", 2023)
//                                                     params {s, L, fast, slow}
void rotary_frequencies(int rot, double base, int scaling, const double* p, uint64_t* freq, float* amplitude) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  double lo = 0, hi = 0;
  *amplitude = 1.f;
  if (scaling == TV_ROPE_BASE) {
    base *= pow(p[0], (double)rot / (rot - 2));
  } else if (scaling == TV_ROPE_YARN) {
    const double a = rot * log(p[1] / (p[2] * kTwoPi)) / (2 * log(base));
    const double z = rot * log(p[1] / (p[3] * kTwoPi)) / (2 * log(base));
    lo = fmax(floor(a), 0.0);
    hi = fmin(ceil(z), rot - 1.0);
    *amplitude = (float)(0.1 * log(p[0]) + 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double r = pow(base, -2.0 * i / rot);
    if (scaling == TV_ROPE_LINEAR) {
      r /= p[0];
    } else if (scaling == TV_ROPE_BANDED) {
      const double m = fmin(fmax((p[3] * r / kTwoPi - p[1]) / (p[2] - p[1]), 0.0), 1.0);
      r *= m + (1.0 - m) / p[0];
    } else if (scaling == TV_ROPE_YARN) {
      const double k = 1.0 - fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
      r *= k + (1.0 - k) / p[0];
    }
    freq[i] = (uint64_t)llrint(r / kTwoPi * 0x1p62) << 2;  // r <= 1: at most 2^62 / 2 pi
  }
}

}  // namespace tv
