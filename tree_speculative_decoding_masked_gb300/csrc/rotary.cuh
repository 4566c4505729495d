// What the kernels that turn heads share (the mathematics: rotary.cu): loads and stores of columns, sines
// and cosines, a token's place, and the norm of a head.
#pragma once

#include "paged.cuh"

namespace tv {

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

// Where token (b, t) sits, and where its row goes in a page (page_row < 0: nowhere).
struct RotPlace {
  long long pos, page_row;
  bool live;
};
__device__ __forceinline__ RotPlace rot_place(const RotaryArgs& a, long long token, int b, int t, bool first,
                                              bool pages) {
  RotPlace r{0, -1, false};
  if (a.table && t == 0 && first) {  // counts and lengths, also where no row is active
    const int n = a.n_rows ? a.n_rows[b] : 0;
    if (n < 0 || n > a.N || a.base[b] < 0) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
  }
  const int off = a.pos ? a.pos[token] : t;
  if (off < 0) return r;  // padding
  const int base = a.base ? a.base[b] : 0;
  if (a.n_rows && (t >= a.n_rows[b] || a.n_rows[b] > a.N)) return r;
  r.pos = (long long)base + off;
  if (pages) {
    const long long row = (long long)base + t;
    const long long pg = row >> a.page_shift;
    const int page = base >= 0 && pg < a.max_pages ? a.table[(size_t)b * a.max_pages + pg] : -1;
    if (page >= 0 && page < a.num_pages)
      r.page_row = ((long long)page * a.Hkv << a.page_shift) + (row & ((1 << a.page_shift) - 1));
    else
      set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
  }
  r.live = r.pos >= 0;  // a negative base
  return r;
}

// x and y over the head's root mean square, times the weight: `part` 0 queries, 1 keys
template <typename T, int kVec>
__device__ __forceinline__ void rot_norm(const RotaryArgs& a, int part, int ea, int eb, bool two, int cols,
                                         uint32_t peers, float (&x)[kVec], float (&y)[kVec]) {
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < kVec; ++k) ss = fmaf(x[k], x[k], fmaf(y[k], y[k], ss));
  for (int o = 1; o < cols; o *= 2) ss += __shfl_xor_sync(peers, ss, o);
  const float r = 1.f / sqrtf(ss / a.D + a.eps);
  const T* weight = reinterpret_cast<const T*>(a.weight[part]);
  using Raw = typename RotRaw<T, kVec>::type;
  float w[kVec];
  rot_unpack<T, kVec>(__ldg(reinterpret_cast<const Raw*>(weight + ea)), w);
#pragma unroll
  for (int k = 0; k < kVec; ++k) x[k] = x[k] * r * w[k];
  if (!two) return;
  rot_unpack<T, kVec>(__ldg(reinterpret_cast<const Raw*>(weight + eb)), w);
#pragma unroll
  for (int k = 0; k < kVec; ++k) y[k] = y[k] * r * w[k];
}

}  // namespace tv
