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
// heads of its group, three heads' loads in flight at a time; the groups are sized so that
// small batches still fill the device.  268 MB (4 x 4096 rows of 32 heads of 128 bf16): 45.9 us,
// 5.85 TB/s of the 6.78 that a copy reaches; four heads a batch and 3 blocks an SM 50.5, two
// and 6 blocks 73.8; half as many groups 47.7, twice as many 56.2.  64 tokens: 2.7 us.
#include <math.h>

#include "paged.cuh"

namespace tv {

constexpr int kRotThreads = 256;
constexpr int kRotHeads = 3;  // heads whose loads are in flight together
constexpr long long kRotBlocks = 152 * 16;  // blocks up to which a token's heads go to separate ones

// kVec contiguous elements in one load or store
template <typename T, int kVec>
struct RotRaw {
  using type = uint4;
};
template <typename T>
struct RotRaw<T, 1> {
  using type = T;
};
template <typename T, int kVec>
__device__ __forceinline__ void rot_unpack(const typename RotRaw<T, kVec>::type& r, float (&f)[kVec]) {
  if constexpr (kVec == 1) {
    if constexpr (sizeof(T) == 2)
      f[0] = bf16_to_f32(r);
    else
      f[0] = r;
  } else {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        f[i] = __uint_as_float(w[i]);
      }
    }
  }
}
template <typename T, int kVec>
__device__ __forceinline__ typename RotRaw<T, kVec>::type rot_pack(const float (&f)[kVec]) {
  if constexpr (kVec == 1) {
    if constexpr (sizeof(T) == 2)
      return (T)(ptx::cvt_bf16x2(f[0], 0.f) & 0xffffu);
    else
      return f[0];
  } else if constexpr (sizeof(T) == 2) {
    return make_uint4(ptx::cvt_bf16x2(f[0], f[1]), ptx::cvt_bf16x2(f[2], f[3]), ptx::cvt_bf16x2(f[4], f[5]),
                      ptx::cvt_bf16x2(f[6], f[7]));
  } else {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
}

// sin and cos of an angle in 2^-64 turns.  The nearest quarter turn goes exactly (integers);
// what is left, at most pi / 4, goes through the Taylor polynomials of degree 9 and 8, off by
// less than 2e-9 and 3e-8.
__device__ __forceinline__ float2 sincos_turns(uint64_t turns) {
  const uint32_t quarter = (uint32_t)((turns + (1ull << 61)) >> 62);
  const float x = (float)(int32_t)((turns - ((uint64_t)quarter << 62)) >> 32) * 1.4629180792671596e-09f;  // 2 pi 2^-32
  const float z = x * x;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);  // 1 / 9!, -1 / 7!
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  s = fmaf(x * z, s, x);
  float c = fmaf(z, 2.4801587e-5f, -1.3888889e-3f);  // 1 / 8!, -1 / 6!
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const float sn = quarter & 1 ? c : s, cs = quarter & 1 ? s : c;
  return make_float2(quarter & 2 ? -sn : sn, (quarter + 1) & 2 ? -cs : cs);
}

// Grid: x over (token, column) pairs, y over groups of `hg` of the Hq + 2 Hkv heads.  A column
// is kVec pairs (rotated part) or up to 2 kVec elements behind it.
template <typename T, int kVec>
__global__ void __launch_bounds__(kRotThreads, 4) rotary_kernel(RotaryArgs a, int cols, int rot_cols, int hg) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const long long id = (long long)blockIdx.x * kRotThreads + threadIdx.x;
  const long long token = id / cols;
  if (token >= (long long)a.B * a.N) return;
  const int col = (int)(id - token * cols);
  const int b = (int)(token / a.N), t = (int)(token - (long long)b * a.N);
  if (a.table && t == 0 && col == 0 && blockIdx.y == 0) {  // counts and lengths, also where no row is active
    const int n = a.n_rows ? a.n_rows[b] : 0;
    if (n < 0 || n > a.N || a.base[b] < 0) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
  }
  const int off = a.pos ? a.pos[token] : t;
  if (off < 0) return;  // padding
  const int base = a.base ? a.base[b] : 0;
  if (a.n_rows && (t >= a.n_rows[b] || a.n_rows[b] > a.N)) return;
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
  // this thread's elements: ea.. and eb.. (eb >= D: none)
  const bool turn = col < rot_cols;
  const bool pairs_inside = a.interleaved && kVec > 1;  // x and y hold kVec / 2 whole pairs each
  int ea, eb;
  if (turn) {
    ea = a.interleaved && kVec == 1 ? 2 * col : kVec * col;
    eb = a.interleaved && kVec == 1 ? ea + 1 : ea + a.rot / 2;
  } else {
    ea = a.rot + kVec * (col - rot_cols);
    eb = ea + kVec * (cols - rot_cols);
  }
  float cs[kVec], sn[kVec];
  if (turn && h0 < a.Hq + a.Hkv) {
#pragma unroll
    for (int u = 0; u < kVec; ++u) {
      int pair = kVec * col + u;
      if (pairs_inside) pair = (u < kVec / 2 ? 0 : a.rot / 4 - kVec / 2) + kVec / 2 * col + u;
      const float2 sc = sincos_turns((uint64_t)p * a.freq[pair]);
      sn[u] = sc.x * a.amplitude;
      cs[u] = sc.y * a.amplitude;
    }
  }
  auto source = [&](int h) -> const T* {
    const int part = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2;
    const int hh = part == 0 ? h : part == 1 ? h - a.Hq : h - a.Hq - a.Hkv;
    return reinterpret_cast<const T*>(a.src[part]) + b * a.sb[part] + hh * a.sh[part] + t * a.sn[part];
  };
  auto target = [&](int h) -> T* {
    if (h < a.Hq) return reinterpret_cast<T*>(a.q_out) + (((long long)b * a.Hq + h) * a.N + t) * a.D;
    if (page_row < 0) return nullptr;
    const bool is_v = h >= a.Hq + a.Hkv;
    const int hh = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
    return reinterpret_cast<T*>(is_v ? a.v_cache : a.k_cache) + (page_row + ((long long)hh << a.page_shift)) * a.D;
  };
  const bool two = eb < a.D;
  using Raw = typename RotRaw<T, kVec>::type;
  for (int hb = h0; hb < h1; hb += kRotHeads) {
    // the batch's loads first: they are in flight together (a row may be rotated in place, so the
    // compiler would not move a load past an earlier head's store)
    Raw ra[kRotHeads], rb[kRotHeads];
#pragma unroll
    for (int u = 0; u < kRotHeads; ++u)
      if (hb + u < h1) {
        const T* src = source(hb + u);
        ra[u] = *reinterpret_cast<const Raw*>(src + ea);
        if (two) rb[u] = *reinterpret_cast<const Raw*>(src + eb);
      }
#pragma unroll
    for (int u = 0; u < kRotHeads; ++u) {
      if (hb + u >= h1) break;
      T* dst = target(hb + u);
      if (!dst) continue;
      if (turn && hb + u < a.Hq + a.Hkv) {
        float x[kVec], y[kVec];
        rot_unpack<T, kVec>(ra[u], x);
        rot_unpack<T, kVec>(rb[u], y);
        if (pairs_inside) {
#pragma unroll
          for (int k = 0; k < kVec / 2; ++k) {
            const float e0 = x[2 * k], o0 = x[2 * k + 1], e1 = y[2 * k], o1 = y[2 * k + 1];
            x[2 * k] = e0 * cs[k] - o0 * sn[k];
            x[2 * k + 1] = o0 * cs[k] + e0 * sn[k];
            y[2 * k] = e1 * cs[kVec / 2 + k] - o1 * sn[kVec / 2 + k];
            y[2 * k + 1] = o1 * cs[kVec / 2 + k] + e1 * sn[kVec / 2 + k];
          }
        } else {
#pragma unroll
          for (int k = 0; k < kVec; ++k) {
            const float e = x[k], o = y[k];
            x[k] = e * cs[k] - o * sn[k];
            y[k] = o * cs[k] + e * sn[k];
          }
        }
        ra[u] = rot_pack<T, kVec>(x);
        rb[u] = rot_pack<T, kVec>(y);
      }
      // values and the elements behind the rotated part go through unchanged (a NaN's bits survive)
      *reinterpret_cast<Raw*>(dst + ea) = ra[u];
      if (two) *reinterpret_cast<Raw*>(dst + eb) = rb[u];
    }
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
  while (hg < heads && blocks * ((heads + hg - 1) / hg) > kRotBlocks) hg *= 2;
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
