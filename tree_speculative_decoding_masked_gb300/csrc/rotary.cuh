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

// 16 bytes and their pair partners of a head as pairs (a[u], b[u]): element u of each of them, or, where neighbours
// turn together, an element and the next.  Two pairs to a word, for arithmetic that takes two numbers at once.
template <int kVec, bool kInter>
__device__ __forceinline__ void rot_to_pairs(const float (&x)[kVec], const float (&y)[kVec], float2 (&a)[kVec / 2],
                                             float2 (&b)[kVec / 2]) {
#pragma unroll
  for (int k = 0; k < kVec / 2; ++k) {
    if constexpr (kInter) {
      const float* f = k < kVec / 4 ? x + 4 * k : y + 4 * (k - kVec / 4);
      a[k] = make_float2(f[0], f[2]), b[k] = make_float2(f[1], f[3]);
    } else {
      a[k] = make_float2(x[2 * k], x[2 * k + 1]), b[k] = make_float2(y[2 * k], y[2 * k + 1]);
    }
  }
}
template <int kVec, bool kInter>
__device__ __forceinline__ void rot_from_pairs(const float2 (&a)[kVec / 2], const float2 (&b)[kVec / 2], float (&x)[kVec],
                                               float (&y)[kVec]) {
#pragma unroll
  for (int k = 0; k < kVec / 2; ++k) {
    if constexpr (kInter) {
      float* f = k < kVec / 4 ? x + 4 * k : y + 4 * (k - kVec / 4);
      f[0] = a[k].x, f[1] = b[k].x, f[2] = a[k].y, f[3] = b[k].y;
    } else {
      x[2 * k] = a[k].x, x[2 * k + 1] = a[k].y, y[2 * k] = b[k].x, y[2 * k + 1] = b[k].y;
    }
  }
}
// the number of pair u of column `col`
template <int kVec, bool kInter>
__device__ __forceinline__ int rot_pair(int rot, int col, int u) {
  return kInter ? (u < kVec / 2 ? 0 : rot / 4 - kVec / 2) + kVec / 2 * col + u : kVec * col + u;
}
// What a row's pairs are multiplied by, the norm's weight taken in: (a, b) -> (a ca + b nb, b cb + a sa).  Once
// for all the heads that a thread turns.
template <int kVec>
struct RotTurn {
  float2 ca[kVec / 2], nb[kVec / 2], cb[kVec / 2], sa[kVec / 2];
};
// w: the weights of the pairs (1 without a norm); columns that do not turn use ca and cb alone
template <int kVec, bool kInter>
__device__ __forceinline__ void rot_turn_set(const RotaryArgs& a, long long pos, bool turn, int col,
                                             const float2 (&wa)[kVec / 2], const float2 (&wb)[kVec / 2],
                                             RotTurn<kVec>& t) {
#pragma unroll
  for (int k = 0; k < kVec / 2; ++k) {
    t.ca[k] = wa[k], t.cb[k] = wb[k];
    if (!turn) continue;
    const float2 p = sincos_turns((uint64_t)pos * a.freq[rot_pair<kVec, kInter>(a.rot, col, 2 * k)]);
    const float2 q = sincos_turns((uint64_t)pos * a.freq[rot_pair<kVec, kInter>(a.rot, col, 2 * k + 1)]);
    const float2 sn = make_float2(p.x * a.amplitude, q.x * a.amplitude);
    const float2 cs = make_float2(p.y * a.amplitude, q.y * a.amplitude);
    t.sa[k] = __fmul2_rn(wa[k], sn);
    t.nb[k] = __fmul2_rn(wb[k], make_float2(-sn.x, -sn.y));
    t.ca[k] = __fmul2_rn(wa[k], cs);
    t.cb[k] = __fmul2_rn(wb[k], cs);
  }
}
template <int kVec>
__device__ __forceinline__ float rot_squares(const float2 (&a)[kVec / 2], const float2 (&b)[kVec / 2]) {
  float2 s = __fmul2_rn(a[0], a[0]);
#pragma unroll
  for (int k = 1; k < kVec / 2; ++k) s = __ffma2_rn(a[k], a[k], s);
#pragma unroll
  for (int k = 0; k < kVec / 2; ++k) s = __ffma2_rn(b[k], b[k], s);
  return s.x + s.y;
}
// r: 1 over the head's root mean square (normed), else unread
template <int kVec>
__device__ __forceinline__ void rot_turn(const RotTurn<kVec>& t, bool normed, float r, bool turn, float2 (&a)[kVec / 2],
                                         float2 (&b)[kVec / 2]) {
  if (normed) {
#pragma unroll
    for (int k = 0; k < kVec / 2; ++k) {
      a[k] = __fmul2_rn(a[k], make_float2(r, r));
      b[k] = __fmul2_rn(b[k], make_float2(r, r));
    }
  }
  if (turn) {
#pragma unroll
    for (int k = 0; k < kVec / 2; ++k) {
      const float2 x = a[k];
      a[k] = __ffma2_rn(b[k], t.nb[k], __fmul2_rn(x, t.ca[k]));
      b[k] = __ffma2_rn(x, t.sa[k], __fmul2_rn(b[k], t.cb[k]));
    }
  } else if (normed) {
#pragma unroll
    for (int k = 0; k < kVec / 2; ++k) a[k] = __fmul2_rn(a[k], t.ca[k]), b[k] = __fmul2_rn(b[k], t.cb[k]);
  }
}

}  // namespace tv
