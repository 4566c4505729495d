// Paged KV caches: page lookup, visibility of keys, and the division of attention work over
// CTAs that the paged attention kernels share.
//
// A cache holds pages [num_pages][Hkv][page_size][D]; cache row r of sequence b is row
// r mod page_size of page page_table[b][r / page_size].  Sequence b's committed rows are
// 0..P_b-1 (P_b = prefix_len[b]) and its new rows P_b..P_b+n_b-1.
#pragma once

#include <cuda.h>

#include "tv_kernels.cuh"
#include "tv_ptx.cuh"

namespace tv {

// New rows of sequence b that the call looks at: n_rows[b] (N without n_rows), or 0 for a sequence with a
// row that does not fit its page table (*bad).  A padded tree's inactive rows need no place: its rows
// count up to the table's end, and paged_cut looks at the first behind it.
__device__ __forceinline__ int paged_rows(const PagedAttn& a, int b, int P, bool* bad) {
  const int n = a.n_rows ? a.n_rows[b] : a.N, room = max((a.max_pages << a.page_shift) - max(P, 0), 0);
  const int m = a.parent ? min(n, room) : n;
  const bool fits = P >= 0 && n >= 0 && n <= a.N && m <= room && (m > 0 || n == 0);
  *bad = !fits;
  return fits ? m : 0;
}
// Whether the table's end cuts off an active row of a tree.
__device__ __forceinline__ bool paged_cut(const PagedAttn& a, int b, int P, int n) {
  return a.parent && n > 0 && P + n == a.max_pages << a.page_shift && n < (a.n_rows ? a.n_rows[b] : a.N) &&
         a.parent[(size_t)b * a.N + n] != -1;
}

// One CTA's share of the attention work.  The work is cut into units (sequence b, KV head,
// tile of RT query rows) of 'key tiles' (KT keys); the units' tiles laid end to end are
// divided into equal contiguous ranges, one per CTA, so that ragged lengths known only
// on the device load every SM alike.  Query row r of a KV head is head r % G of node
// r / G, so that a row tile spans few nodes and its key range ends at its last one.
struct PagedSpan {
  long long W;      // key tiles in all
  long long per;    // tiles per CTA
  int b;            // where this CTA starts: sequence,
  long long base;   // and that sequence's first tile
  int whole;        // not 0: every unit counts as this many tiles, one unit per CTA
  int tol;          // a cut this near to a unit's edge moves to the edge
  int fix;          // what a unit costs beside its tiles, in tiles: each counts as so many more
};
constexpr int kPagedRed = 34 + 512;  // scratch of paged_span: CTAs of up to 512 threads

__device__ __forceinline__ int unit_rows(const PagedAttn& a, int n, int rt, int RT) {
  return max(0, min(RT, n * a.G - rt * RT));
}
// first key that some row of row tile rt can see (trees: any node may sit at depth 0..)
__device__ __forceinline__ int unit_lo(const PagedAttn& a, int P, int rt, int RT) {
  if (a.window <= 0) return 0;
  const int i = a.parent ? 0 : rt * RT / a.G;
  return max(0, P + i - a.window + 1);
}
__device__ __forceinline__ int unit_tiles(const PagedAttn& a, int P, int n, int rt, int RT, int KT) {
  const int rows = unit_rows(a, n, rt, RT);
  if (rows == 0) return 0;
  const int hi = P + (rt * RT + rows - 1) / a.G + 1;
  return (hi + KT - 1) / KT - unit_lo(a, P, rt, RT) / KT;
}
// Tiles of one KV head of a sequence; a warp's lanes share the sum over its row tiles.
__device__ inline long long head_tiles_warp(const PagedAttn& a, int P, int n, int RT, int KT, int whole, int fix) {
  const int row_tiles = (n * a.G + RT - 1) / RT;
  if (whole) return (long long)whole * row_tiles;
  unsigned long long s = 0;
  for (int rt = threadIdx.x & 31; rt * RT < n * a.G; rt += 32) s += unit_tiles(a, P, n, rt, RT, KT);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return (long long)s + (long long)fix * row_tiles;
}

// Every thread of the CTA calls it; red holds kPagedRed entries.  A CTA takes min_per tiles or more.
// kWhole: where the units are at most the CTAs and the longest is little longer than an equal share (by
// a quarter and 8 tiles, or 30), each CTA takes one unit whole instead: no merge, and at the power limit
// more busy SMs only clock lower.  128 units on 152 SMs, whole / cut: 16 x 64 nodes over 1000 tokens
// 29.8 / 45.2 us, over 4000 70.0 / 80.2, 8 x 128 nodes over 8000 120 / 126 (cut by the rule from 11600 on);
// 80 units over 1000 tokens 30.5 / 33.3 (from 3500 on).
template <bool kWhole = false>
__device__ inline PagedSpan paged_span(const PagedAttn& a, int RT, int KT, int min_per, unsigned long long* red,
                                       int tol = 0, int fix = 0) {
  PagedSpan sp;
  sp.whole = 0;
  sp.tol = tol;
  sp.fix = fix;
  unsigned long long W = 0, mine = 0, at = 0;
  bool any_bad = false;
  // tiles of sequence b0 + threadIdx.x: by its own thread, or with many row tiles a warp each
  const bool many = a.N * a.G > 4 * RT;
  auto tiles_of = [&](int b0) -> unsigned long long {
    const int b = b0 + threadIdx.x;
    unsigned long long t = 0;
    if (many) {
      const int count = min((int)blockDim.x, a.B - b0);
      for (int k = threadIdx.x >> 5; k < count; k += blockDim.x >> 5) {
        const int P = a.prefix_len[b0 + k];
        bool bad = false;
        const int n = paged_rows(a, b0 + k, P, &bad);
        any_bad |= bad || paged_cut(a, b0 + k, P, n);
        const long long head = head_tiles_warp(a, P, n, RT, KT, sp.whole, fix);
        if ((threadIdx.x & 31) == 0) red[34 + k] = (unsigned long long)head;
      }
      __syncthreads();
      if (b < a.B) t = red[34 + threadIdx.x] * a.Hkv;
    } else if (b < a.B) {
      const int P = a.prefix_len[b];
      bool bad = false;
      const int n = paged_rows(a, b, P, &bad);
      any_bad |= bad || paged_cut(a, b, P, n);
      for (int rt = 0; rt * RT < n * a.G; ++rt) t += sp.whole ? sp.whole : unit_tiles(a, P, n, rt, RT, KT) + fix;
      t *= a.Hkv;
    }
    return t;
  };
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    mine = tiles_of(b0);
    unsigned long long part = 0;
    at = W + block_scan_u64(mine, red, &part);
    W += part;
  }
  if (any_bad && blockIdx.x == 0) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
  sp.W = (long long)W;
  sp.per = max((long long)min_per, (sp.W + gridDim.x - 1) / gridDim.x);
  if constexpr (kWhole) {
    unsigned long long units = 0, longest = 0;
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
      const int P = a.prefix_len[b];
      bool bad = false;
      const int n = paged_rows(a, b, P, &bad), rts = (n * a.G + RT - 1) / RT;
      units += (unsigned long long)rts * a.Hkv;
      // a causal or tree row tile sees no more keys than the last, a window bounds them all
      if (rts > 0) longest = max(longest, (unsigned long long)max(unit_tiles(a, P, n, rts - 1, RT, KT),
                                                                  unit_tiles(a, P, n, max(0, rts - 2), RT, KT)));
    }
    unsigned long long all = 0;
    block_scan_u64(units, red, &all);
    if (threadIdx.x == 0) red[0] = 0;
    __syncthreads();
    atomicMax(&red[0], longest);
    __syncthreads();
    longest = red[0];
    __syncthreads();
    if (all <= gridDim.x && longest + fix <= (unsigned long long)(sp.per + min(sp.per / 4 + 8, 30ll))) {
      sp.whole = (int)longest;
      sp.per = sp.whole;
      W = all * longest;
      sp.W = (long long)W;
      mine = tiles_of(0);
      if (a.B <= (int)blockDim.x) {
        unsigned long long part = 0;
        at = block_scan_u64(mine, red, &part);
      }
    }
  }
  const unsigned long long begin = (unsigned long long)sp.per * blockIdx.x;
  sp.b = a.B;
  sp.base = sp.W;
  if (begin >= W) return sp;  // the same for the whole CTA
  // the sequence that holds tile `begin`; with more sequences than threads their tiles are
  // counted once more
  unsigned long long cum = 0;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    unsigned long long part = 0;
    if (a.B > (int)blockDim.x) {
      mine = tiles_of(b0);
      at = cum + block_scan_u64(mine, red, &part);
      cum += part;
    } else {
      cum = W;
    }
    if (begin >= at && begin < at + mine) {
      red[0] = (unsigned long long)(b0 + threadIdx.x);
      red[1] = at;
    }
    __syncthreads();
    if (begin < cum) {
      sp.b = (int)red[0];
      sp.base = (long long)red[1];
      __syncthreads();
      break;
    }
  }
  return sp;
}

// The units of a CTA's range, one after another.  A warp's lanes call unit_next together.
struct UnitWalk {
  long long pos, end, per;  // tiles still to take; tiles per CTA
  long long seq, head;      // first tile of sequence b; tiles of one of its KV heads
  long long u0, u1;         // the unit's tiles
  int b, hk, rt, P, n;      // the unit; the sequence's committed and new rows
  int t0, t1;               // of the unit's tiles, those to take
  int loaded, whole, tol, fix;
  bool begun;
};

// a / b of numbers >= 0, in 32 bits where they fit
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}
// How near to the left (.x) and right edge of a unit of U tiles a cut moves to it.  Units no longer than
// a CTA's share: tol, or half the unit.  Longer ones are cut anyhow, and moved cuts only unbalance
// the ranges: what leaves next to no tiles on one side.
__device__ __forceinline__ int2 unit_tol(long long U, long long per, int tol, int fix) {
  const long long l = U <= per ? tol : min(tol, fix + 2), r = U <= per ? tol : min(tol, 4);
  return make_int2((int)min(l, U / 2), (int)min(r, (U - 1) / 2));
}
// Where the boundary p of two ranges, strictly inside unit [u0, u1), cuts it.
__device__ __forceinline__ long long unit_cut(long long p, long long u0, long long u1, const UnitWalk& w) {
  const int2 tol = unit_tol(u1 - u0, w.per, w.tol, w.fix);
  return p - u0 <= tol.x ? u0 : u1 - p <= tol.y ? u1 : p;
}
// The CTAs c0..c1 that share the walk's unit; c1 <= c0 where none cuts it.
struct UnitCtas {
  long long c0, c1;
};
__device__ __forceinline__ UnitCtas unit_ctas(const UnitWalk& w) {
  const int2 tol = unit_tol(w.u1 - w.u0, w.per, w.tol, w.fix);
  return {div_ll(w.u0 + tol.x, w.per), div_ll(w.u1 - tol.y - 1, w.per)};
}
__device__ __forceinline__ UnitWalk unit_walk(const PagedSpan& sp) {
  UnitWalk w{};
  w.per = max(1ll, sp.per);  // sp.per: 0 where no row is active
  w.pos = sp.per * blockIdx.x;
  w.end = min(sp.W, w.pos + sp.per);
  w.seq = sp.base;
  w.b = sp.b;
  w.loaded = -1;
  w.whole = sp.whole;
  w.tol = sp.tol;
  w.fix = sp.fix;
  return w;
}
__device__ inline bool unit_next(const PagedAttn& a, UnitWalk& w, int RT, int KT) {
  const int lane = threadIdx.x & 31;
  while (w.pos < w.end && w.b < a.B) {
    if (w.loaded != w.b) {
      bool bad;
      w.P = a.prefix_len[w.b];
      w.n = paged_rows(a, w.b, w.P, &bad);
      w.head = head_tiles_warp(a, w.P, w.n, RT, KT, w.whole, w.fix);
      w.loaded = w.b;
    }
    long long rel = w.pos - w.seq;
    if (rel >= w.head * a.Hkv) {
      w.seq += w.head * a.Hkv;
      ++w.b;
      continue;
    }
    w.hk = (int)div_ll(rel, w.head);
    rel -= w.hk * w.head;
    for (int rt0 = 0;; rt0 += 32) {  // ends: rel lies below the head's sum
      unsigned t = unit_tiles(a, w.P, w.n, rt0 + lane, RT, KT);
      if (t) t = w.whole ? w.whole : t + w.fix;
      unsigned incl = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned total = __shfl_sync(0xffffffffu, incl, 31);
      if (rel >= (long long)total && (rt0 + 32) * RT < w.n * a.G) {
        rel -= total;
        continue;
      }
      const int k = max(0, __ffs(__ballot_sync(0xffffffffu, (long long)incl > rel)) - 1);
      const unsigned T = __shfl_sync(0xffffffffu, t, k), upto = __shfl_sync(0xffffffffu, incl, k);
      w.rt = rt0 + k;
      w.u0 = w.pos - (rel - (long long)(upto - T));
      w.u1 = w.u0 + T;
      break;
    }
    if (!w.begun) {
      w.begun = true;
      if (w.pos > w.u0) w.pos = unit_cut(w.pos, w.u0, w.u1, w);
      if (w.pos == w.u1) continue;
    }
    long long end = w.u1;
    if (w.end < w.u1) end = unit_cut(w.end, w.u0, w.u1, w);
    if (end <= w.pos) return false;
    w.t0 = max(0, (int)(w.pos - w.u0) - w.fix);
    w.t1 = max(0, (int)(end - w.u0) - w.fix);
    w.pos = end;
    if (w.whole) w.t1 = unit_tiles(a, w.P, w.n, w.rt, RT, KT);
    return true;
  }
  return false;
}

// Of a cut unit [u0, u1), CTA c parks its partial result in slot 2c if the unit begins before the
// CTA's range and in slot 2c + 1 if not: a CTA has one piece that a cut begins and one that a cut ends,
// and if its range's first cut has moved to u0, none that a cut begins.  The unit's counter is
// that of its first CTA (a CTA is the first of one cut unit at most).
__device__ __forceinline__ int unit_slot(long long c, long long per, long long u0) {
  return (int)(2 * c + (u0 < c * per ? 0 : 1));
}

// How scores are capped in the bf16 kernels: not at all; by soft_tanh; or, past kPlainCap, by capped_score.
// soft_tanh is off by some 2^-22 of 1 however small its argument, and a score by that times the cap:
// at 256 a weight by 2^-14, little beside its rounding to bf16.  Two chunks of 2048 rows over 3000 to 6000
// tokens: 519 us by soft_tanh4, 692 by the series; one token each of 32 sequences 126 by either.
enum { kNoCap, kTanhCap, kLargeCap };
constexpr float kPlainCap = 256.f;
inline int cap_mode(float cap) { return cap > kPlainCap ? kLargeCap : cap > 0.f ? kTanhCap : kNoCap; }

// tanh(y / 2) with y given as x = y log2 e: 1 - 2 / (1 + 2^x), off by an ulp or two of 1
__device__ __forceinline__ float soft_tanh(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ptx::ex2(x)));
  return fmaf(-2.f, r, 1.f);
}

// (tanh x - x) / x^3 for z = x^2 below 0.45^2: the Taylor series up to x^13 (the next term is 2^-25 of x)
__device__ __forceinline__ float tanh_tail(float z) {
  float p = fmaf(z, 3.5921280e-3f, -8.8632355e-3f);  // 21844 / 6081075, -1382 / 155925
  p = fmaf(z, p, 2.1869489e-2f);                     // 62 / 2835
  p = fmaf(z, p, -5.3968254e-2f);                    // -17 / 315
  p = fmaf(z, p, 1.3333333e-1f);
  return fmaf(z, p, -3.3333333e-1f);
}
constexpr float kTanhNear = 0.2025f;

// tanh to an ulp or two: the series below 0.45, where capped scores mostly lie, else the library's
__device__ __forceinline__ float tanh_f32(float x) {
  const float z = x * x;
  if (z >= kTanhNear || isnan(x)) return tanhf(x);
  return fmaf(x * z, tanh_tail(z), x);
}

// cap tanh(t / cap) to some 2^-21 of itself, at any cap: below 0.45 cap the series as a correction of t
__device__ __forceinline__ float capped_score(float t, float cap, float inv_cap) {
  const float x = t * inv_cap, z = x * x;
  const float far = cap * soft_tanh(x * (2.f * kLog2e));
  return z >= kTanhNear ? far : fmaf(t * z, tanh_tail(z), t);
}

// the smaller of the two, NaN where x is
__device__ __forceinline__ float min_nan(float x, float y) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// four soft_tanh with one reciprocal: 1 / a = (1 / abcd) (b cd).  2^x is held below 2^30, where tanh
// has long been 1, so the product stays finite.  A NaN makes its neighbours NaN: the caller zeroes the
// scores of keys that may not be seen, whose rows may hold anything, so that only a NaN query does.
__device__ __forceinline__ void soft_tanh4(float* s, float k) {
  // two an instruction where the hardware has it: 545 -> 539 us for two chunks of 2048 rows
  const float2 kk = make_float2(k, k), one = make_float2(1.f, 1.f);
  const float2 x0 = __fmul2_rn(make_float2(s[0], s[1]), kk), x1 = __fmul2_rn(make_float2(s[2], s[3]), kk);
  const float2 a0 = __fadd2_rn(make_float2(ptx::ex2(min_nan(x0.x, 30.f)), ptx::ex2(min_nan(x0.y, 30.f))), one);
  const float2 a1 = __fadd2_rn(make_float2(ptx::ex2(min_nan(x1.x, 30.f)), ptx::ex2(min_nan(x1.y, 30.f))), one);
  const float ab = a0.x * a0.y, cd = a1.x * a1.y;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ab * cd));
  const float2 q = __fmul2_rn(make_float2(cd, ab), make_float2(-2.f * r, -2.f * r));
  const float2 t0 = __ffma2_rn(make_float2(q.x, q.x), make_float2(a0.y, a0.x), one);
  const float2 t1 = __ffma2_rn(make_float2(q.y, q.y), make_float2(a1.y, a1.x), one);
  s[0] = t0.x, s[1] = t0.y, s[2] = t1.x, s[3] = t1.y;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_addr(dst)), "l"(src) : "memory");
}

// ---- host side
constexpr int kPagedMaxSms = 160;  // sizes the workspaces
constexpr int kPagedMaxCtas = 2;   // CTAs per SM of the largest persistent grid
constexpr size_t kPagedCntBytes = kPagedMaxCtas * kPagedMaxSms * 4;
constexpr int kPagedFewRows = 16;  // query rows of a KV head above which row tiles are used

int paged_device_sms();
bool paged_tc_takes(int Hq, int Hkv, int D, int N);
PagedWs paged_tc_ws(int B, int Hq, int Hkv, int D, int N);
cudaError_t launch_paged_tc(PagedAttn a, char* ws, cudaStream_t stream);
PagedWs paged_mma_ws(int B, int Hq, int Hkv, int D, int N, int sms);
cudaError_t launch_paged_mma(PagedAttn a, char* ws, cudaStream_t stream);
PagedWs paged_f32_ws(int B, int Hq, int Hkv, int D, int N);
cudaError_t launch_paged_f32(PagedAttn a, char* ws, cudaStream_t stream);
PagedWs paged_simt_ws(int D);
cudaError_t launch_paged_simt(PagedAttn a, char* ws, cudaStream_t stream);
// Tensor map of bf16 pages, 128-byte swizzle.  D = 128 and 256: 5-D, a box spans all column
// blocks and min(page_size, 64) rows, as 8-row groups [block][8][128 bytes].  Other D: 3-D boxes
// of one column block, of min(page_size, 64) rows (D <= 64) or 8.
bool paged_kv_tmap(CUtensorMap* m, const void* base, const PagedAttn& a);

}  // namespace tv
