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

#include "rotary.cuh"

namespace tv {

constexpr int kRotThreads = 256;
constexpr int kRotHeads = 3;  // heads whose loads are in flight together
constexpr long long kRotBlocks = 152 * 16;  // blocks up to which a token's heads go to separate ones
constexpr int kNormHeads = 3;               // the same two with norms
constexpr long long kNormBlocks = 152 * 8;

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
  const int heads = a.Hq + 2 * a.Hkv;
  const int h0 = blockIdx.y * hg, h1 = min(heads, h0 + hg);
  const RotPlace at = rot_place(a, token, b, t, col == 0 && blockIdx.y == 0, h1 > a.Hq);
  if (!at.live) return;
  const long long p = at.pos, page_row = at.page_row;
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

// The same with norms: queries and keys are first divided by their root mean square over the head and multiplied
// by a weight, in 32 bits.  The `cols` (a power of two up to 32) threads of a token are neighbours in a warp and add
// up their squares by shuffles; the weight goes into the sines and cosines, which a thread takes once for its
// group's heads, all of them queries, keys or values, and the arithmetic is two numbers an instruction.  268 MB (4 x
// 4096 rows of 32 heads of 128 bf16, 64 turned): 51.8 us, 5.2 TB/s; two heads in flight 53.3, four 58.7 (spills); four
// that are not loaded ahead of the work on those before 54.5, two of them 66; with a branch a head 75.  64 tokens: 3.3 us.
template <typename T, int kVec, bool kInter>
__global__ void __launch_bounds__(kRotThreads, 2) norm_rotary_kernel(RotaryArgs a, int cols, int rot_cols, int hg) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int col = threadIdx.x & (cols - 1);
  const long long token = (long long)blockIdx.x * (kRotThreads / cols) + threadIdx.x / cols;
  if (token >= (long long)a.B * a.N) return;
  const int b = (int)token / a.N, t = (int)token - b * a.N;  // kMaxRotaryRows fits an int
  const int qg = (a.Hq + hg - 1) / hg, kg = (a.Hkv + hg - 1) / hg;
  const int part = (int)blockIdx.y < qg ? 0 : (int)blockIdx.y < qg + kg ? 1 : 2;
  const int h0 = ((int)blockIdx.y - (part == 0 ? 0 : part == 1 ? qg : qg + kg)) * hg;
  const int heads = min(part ? a.Hkv : a.Hq, h0 + hg) - h0;
  const RotPlace at = rot_place(a, token, b, t, col == 0 && blockIdx.y == 0, part > 0);
  if (!at.live || (part > 0 && at.page_row < 0)) return;
  const bool turn = col < rot_cols && part < 2;
  const int ea = col < rot_cols ? kVec * col : a.rot + kVec * (col - rot_cols);
  const int eb = ea + (col < rot_cols ? a.rot / 2 : kVec * (cols - rot_cols));
  using Raw = typename RotRaw<T, kVec>::type;
  // the loads of heads h and on, kNormHeads of them or one, ahead of the work on those before
  const long long sh = a.sh[part];
  const T* src = reinterpret_cast<const T*>(a.src[part]) + b * a.sb[part] + h0 * sh + t * a.sn[part];
  Raw ra[kNormHeads], rb[kNormHeads];
  auto load = [&](int h) {
    const T* from = src + h * sh;
    if (h + kNormHeads <= heads) {
#pragma unroll
      for (int u = 0; u < kNormHeads; ++u) {
        ra[u] = *reinterpret_cast<const Raw*>(from + u * sh + ea);
        rb[u] = *reinterpret_cast<const Raw*>(from + u * sh + eb);
      }
    } else if (h < heads) {
      ra[0] = *reinterpret_cast<const Raw*>(from + ea);
      rb[0] = *reinterpret_cast<const Raw*>(from + eb);
    }
  };
  load(0);
  RotTurn<kVec> turns;
  if (part < 2) {
    const T* weight = reinterpret_cast<const T*>(a.weight[part]);
    float x[kVec], y[kVec];
    rot_unpack<T, kVec>(*reinterpret_cast<const Raw*>(weight + ea), x);
    rot_unpack<T, kVec>(*reinterpret_cast<const Raw*>(weight + eb), y);
    float2 wa[kVec / 2], wb[kVec / 2];
    rot_to_pairs<kVec, kInter>(x, y, wa, wb);
    rot_turn_set<kVec, kInter>(a, at.pos, turn, col, wa, wb, turns);
  }
  const long long step = part ? (long long)a.D << a.page_shift : (long long)a.N * a.D;  // a head's, of the target
  T* dst = part == 0 ? reinterpret_cast<T*>(a.q_out) + (((long long)b * a.Hq + h0) * a.N + t) * a.D
                     : reinterpret_cast<T*>(part == 1 ? a.k_cache : a.v_cache) +
                           (at.page_row + ((long long)h0 << a.page_shift)) * a.D;
  const uint32_t peers = cols == 32 ? ~0u : ((1u << cols) - 1u) << (threadIdx.x & 31 & -cols);
  const float inv_d = 1.f / a.D;
  // heads h.., which have been loaded, without a branch among them
  auto turn_heads = [&](auto many, int h) {
    constexpr int kMany = decltype(many)::value;
    float2 pa[kMany][kVec / 2], pb[kMany][kVec / 2];
    float ss[kMany];
#pragma unroll
    for (int u = 0; u < kMany; ++u) {
      float x[kVec], y[kVec];
      rot_unpack<T, kVec>(ra[u], x);
      rot_unpack<T, kVec>(rb[u], y);
      rot_to_pairs<kVec, kInter>(x, y, pa[u], pb[u]);
      ss[u] = rot_squares<kVec>(pa[u], pb[u]);
    }
    load(h + kMany);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      if (o >= cols) continue;
#pragma unroll
      for (int u = 0; u < kMany; ++u) ss[u] += __shfl_xor_sync(peers, ss[u], o);
    }
#pragma unroll
    for (int u = 0; u < kMany; ++u) {
      float x[kVec], y[kVec];
      rot_turn<kVec>(turns, true, __frsqrt_rn(fmaf(ss[u], inv_d, a.eps)), turn, pa[u], pb[u]);
      rot_from_pairs<kVec, kInter>(pa[u], pb[u], x, y);
      *reinterpret_cast<Raw*>(dst + (h + u) * step + ea) = rot_pack<T, kVec>(x);
      *reinterpret_cast<Raw*>(dst + (h + u) * step + eb) = rot_pack<T, kVec>(y);
    }
  };
  if (part == 2) {
    for (int h = 0; h < heads; ++h) {
      const Raw x = *reinterpret_cast<const Raw*>(src + h * sh + ea), y = *reinterpret_cast<const Raw*>(src + h * sh + eb);
      *reinterpret_cast<Raw*>(dst + h * step + ea) = x;
      *reinterpret_cast<Raw*>(dst + h * step + eb) = y;
    }
    return;
  }
  int h = 0;
  for (; h + kNormHeads <= heads; h += kNormHeads) turn_heads(std::integral_constant<int, kNormHeads>(), h);
  for (; h < heads; ++h) turn_heads(std::integral_constant<int, 1>(), h);
}

// The same with norms for heads and rows that norm_rotary_kernel's columns do not fit (no power of two of
// columns, or not 16 bytes each): a warp a row, an element and its pair partner a lane.
template <typename T>
__global__ void __launch_bounds__(kRotThreads) norm_rows_kernel(RotaryArgs a) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, heads = a.Hq + 2 * a.Hkv;
  const long long token = (long long)blockIdx.x * (kRotThreads / 32) + (threadIdx.x >> 5);
  if (token >= (long long)a.B * a.N) return;
  const int b = (int)(token / a.N), t = (int)(token - (long long)b * a.N);
  const RotPlace at = rot_place(a, token, b, t, lane == 0 && blockIdx.y == 0, a.Hkv > 0 && blockIdx.y >= a.Hq);
  if (!at.live) return;
  for (int h = blockIdx.y; h < heads; h += gridDim.y) {
    const int part = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2;
    const int hh = part == 0 ? h : part == 1 ? h - a.Hq : h - a.Hq - a.Hkv;
    if (part && at.page_row < 0) continue;
    const T* src = reinterpret_cast<const T*>(a.src[part]) + b * a.sb[part] + hh * a.sh[part] + t * a.sn[part];
    T* dst = part == 0 ? reinterpret_cast<T*>(a.q_out) + (((long long)b * a.Hq + h) * a.N + t) * a.D
                       : reinterpret_cast<T*>(part == 1 ? a.k_cache : a.v_cache) +
                             (at.page_row + ((long long)hh << a.page_shift)) * a.D;
    if (part == 2) {
      for (int d = lane; d < a.D; d += 32) dst[d] = src[d];
      continue;
    }
    auto num = [](T v) -> float {
      if constexpr (sizeof(T) == 2)
        return bf16_to_f32(v);
      else
        return v;
    };
    auto put = [&](int d, float f) {
      if constexpr (sizeof(T) == 2)
        dst[d] = (T)(ptx::cvt_bf16x2(f, 0.f) & 0xffffu);
      else
        dst[d] = f;
    };
    float ss = 0.f;
    for (int d = lane; d < a.D; d += 32) ss = fmaf(num(src[d]), num(src[d]), ss);
    const float r = 1.f / sqrtf(warp_sum(ss) / a.D + a.eps);
    const T* weight = reinterpret_cast<const T*>(a.weight[part]);
    for (int i = lane; i < a.rot / 2 + (a.D - a.rot); i += 32) {
      if (i >= a.rot / 2) {
        const int d = i + a.rot / 2;
        put(d, num(src[d]) * r * num(weight[d]));
        continue;
      }
      const int d0 = a.interleaved ? 2 * i : i, d1 = a.interleaved ? 2 * i + 1 : i + a.rot / 2;
      const float2 sc = sincos_turns((uint64_t)at.pos * a.freq[i]);
      const float x = num(src[d0]) * r * num(weight[d0]), y = num(src[d1]) * r * num(weight[d1]);
      const float c = sc.y * a.amplitude, s = sc.x * a.amplitude;
      put(d0, x * c - y * s);
      put(d1, y * c + x * s);
    }
  }
}

template <typename T, int kVec>
static cudaError_t launch_norm_rot(const RotaryArgs& a, cudaStream_t stream) {
  const int cols = a.D / (2 * kVec);
  const long long blocks = ((long long)a.B * a.N * cols + kRotThreads - 1) / kRotThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto groups = [&](int g) { return (long long)(a.Hq + g - 1) / g + 2ll * ((a.Hkv + g - 1) / g); };
  int hg = 1;
  while (hg < max(a.Hq, a.Hkv) && blocks * groups(hg) > kNormBlocks) hg *= 2;
  return launch_pdl(a.interleaved ? norm_rotary_kernel<T, kVec, true> : norm_rotary_kernel<T, kVec, false>,
                    dim3((unsigned)blocks, (unsigned)groups(hg)), dim3(kRotThreads), 0, stream, nullptr, 0, a, cols,
                    a.rot / (2 * kVec), hg);
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
  if (a.weight[0] || a.weight[1]) {
    for (const void* p : a.weight) wide = wide && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    const int cols = a.D / (2 * vec);
    // the columns of a head: a power of two up to a warp, none of them half empty
    if (wide && a.D % (2 * vec) == 0 && cols <= 32 && (cols & (cols - 1)) == 0)
      return dtype == TV_BF16 ? launch_norm_rot<uint16_t, 8>(a, stream) : launch_norm_rot<float, 4>(a, stream);
    const long long blocks = ((long long)a.B * a.N + kRotThreads / 32 - 1) / (kRotThreads / 32);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks, (unsigned)(a.Hq + 2 * a.Hkv));
    return launch_pdl(dtype == TV_BF16 ? norm_rows_kernel<uint16_t> : norm_rows_kernel<float>, grid,
                      dim3(kRotThreads), 0, stream, nullptr, 0, a);
  }
  if (dtype == TV_BF16)
    return wide ? launch_rot<uint16_t, 8>(a, stream) : launch_rot<uint16_t, 1>(a, stream);
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
