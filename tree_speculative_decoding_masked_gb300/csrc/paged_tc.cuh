// Attention of new rows over a paged KV cache on the 5th-generation tensor cores (tcgen05,
// TMEM, TMA), for chunks and trees whose rows fill row tiles.
//
//   S = Q K^T,  P = 2^(c S - m) over the visible keys,  O += P V,  out = O / sum P
//
// with the softmax's maximum and sum in 32 bits and P rounded to bf16 for the second product
// (2^-8 of each weight, the tensor core's input type).  One CTA owns two 128-row tiles A and
// B of one (sequence, KV head) - the G query heads of NT = 128 / G nodes each - and streams a
// range of 64-key tiles once for both, so a page fetched from L2 serves 256 rows.
//
// Pages: a tile is fetched in boxes of min(page_size, 64) rows, each by a lane of the producer
// warp from the page that its own table entry names, read ahead.  At D = 128 a box is 5-D
// (64 columns, 8 rows, 2 column halves, row groups of 8): both halves come in one copy, laid
// out as 8-row groups of [half][8 rows][128 bytes], whose group stride of 2 KB the products'
// descriptors carry.  Boxes of 64 columns each would be twice as many, and at 16-row pages
// the copies' issue, not their bytes, set the pace (590 us for eight 128-node trees over
// 32768 tokens against 428 at 64-row pages).  Boxes that hold no needed row are not fetched
// and their table entries not used.  V rows outside the needed range (the tail of a
// sequence's last page, rows behind the window) may hold anything, NaN included, which a
// zero weight would not remove: the PV issuer's warp zeroes them in shared memory first.
//
// Warps: 0 producer (V a tile behind K), 1 S issuer of tile A (loads its Q) and TMEM owner,
// 2-9 softmax (four per tile, one row a thread), 10 PV issuer, 11 S issuer of tile B.
// TMEM columns: S_A[0] 0.., S_A[1] 64.., S_B[0] 128.., S_B[1] 192.., O_A 256.., O_B 384...
// P_X (bf16, 32 columns) overwrites the first half of its own S buffer.
//
// Two schedules.  Where clusters of two or more CTAs hold all row tiles (or pairs) at once, each
// one's keys are cut into equal parts that run as one thread-block cluster and merge behind its
// barrier; a CTA with one tile has half the partial rows to park and merge, which costs a
// short range more than K and V read twice.  Otherwise a persistent grid of one CTA per SM divides
// all pairs' 64-key steps equally (paged.cuh), which keeps ragged batches and causal triangles
// balanced; a pair cut between CTAs is merged through the workspace, in CTA order, by the CTA that
// finishes last.  There the pieces follow one another without a stop: the producer finds each
// and posts it, keeps the rings filled across pieces, and Q and the first scores of the next
// are there when the softmax warps have written a piece out.  With a stop and a fresh set-up
// at each piece, and every warp finding it for itself, 16 chunks of 512 rows over 1000 to 2000
// tokens took 264 us, now 238; two of 2048 rows over 3000 to 6000 326, now 310.
//
// Pages in 8 bits (kQ8, q8.cuh).  S = Q K^T takes K's codes as they are, as e4m3 products: a row of Q,
// times a power of two that brings its largest element to 2^7..2^8, is the sum of two rows of e4m3
// numbers, the nearest ones and the nearest to what those leave, off by 2^-17 of the largest element at most
// (bf16 elements down to 2^-10 of it exactly).  Two products at twice the rate take what one in bf16 did, and
// K's half comes through L2 and shared memory in half the bytes.  A block's scale of K joins the row's
// power of two in the factor that the softmax multiplies by anyhow, one for 16 keys.  V's codes become fp16
// numbers, which hold them exactly (a conversion for two codes), in a second ring, which four converter
// warps fill; they also zero the rows that no row needs, and bring Q and the scales.  fp16's range is not
// that of the numbers, so V's scales stay out of it: with e the exponent of the value block, P = 2^(z + e - m) and m
// is the running reference of z + e, so that P is at most 2^8 (held times 2^7); the sum takes 2^-e times a block's
// P, or, where an e is far from 0 (a block of zeros: q8_far), goes by z alone.  In fp16 P keeps 11 bits down to 2^-14, 2^-21
// of the row's largest term, fewer below, none below 2^-32 of it.  Warps then: 0 producer, 1 S issuer A,
// 2 PV issuer, 3 S issuer B, 4-11 softmax, 12-15 converters, with registers moved from the others to the
// softmax's (168 and 88 a thread).  V in bf16 with its scales, four times the conversion's instructions, and a
// factor a key or 16 keys by a branch in one kernel: eight 128-node trees over 32768 tokens 612 us.  Blocks of less
// than 16 rows have an instance of their own.  These trees take 342 us now (bf16 pages 298), two chunks of 2048 rows over
// 3000 to 6000 413 (302), a 64-node tree over 2048 16.9 (12.7), the trees with one key a block 540 in the second
// instance; with values of zeros throughout 705 and 1260.  A step, 0.66 us, is bound by what the softmax warps and the converters issue, 0.54 of all slots,
// and by instruction fetches: waits in few lines, loops that are not unrolled and one barrier for a tile's K and V
// took the missed lines of a step from 77 to 26 (bf16: 18) and the trees from 386 us.
#pragma once

#include <atomic>
#include <type_traits>

#include "paged.cuh"
#include "q8.cuh"

namespace tv {

constexpr int kPtRows = 128;
constexpr int kPtKeys = 64;
constexpr int kPtSlots = 4;      // K ring and V ring depth
constexpr int kPtVbSlots = 3;    // kQ8: ring of converted V tiles
constexpr int kPtAhead = 4;      // kQ8: tiles that scales are looked up ahead
constexpr int kPtRound = 68;     // kQ8: floats of a round's scales
constexpr int kPtPieces = 4;     // pieces known ahead
constexpr int kPtMaxSplits = 8;  // portable cluster size
// A unit's set-up and end count as 8 steps, and cuts less than 12 from a unit's edge move to it
// (paged.cuh).  0 and 0 / 12 and 0 / 12 and 8: nine causal chunks of 1510 to 1758 rows on empty caches
// 72.5 / 61.3 / 56.2 us, one of 2048 rows 81.5 / 68.2 / 57.9, 64 trees of 16 nodes over 1000 tokens
// 92.7 / 77.0 / 77.4.
constexpr int kPtTol = 12;
constexpr int kPtFix = 8;
constexpr float kPtRescaleLog2 = 8.f;
constexpr float kPtRescaleSum = 256.f;

// What the pages hold: bf16; 8 bits with blocks of 16 rows or more; with shorter blocks.
enum { kPtBf16, kPtQ8, kPtQ8Fine };

template <int D, int kQ>
struct PtCfg {
  static constexpr bool kQ8 = kQ != kPtBf16;
  static constexpr int kThreads = kQ8 ? 512 : 384;
  static constexpr int kDB = D / 64;
  // bytes per 64-column block of one Q tile; kQ8: per e4m3 part, 128-byte rows
  static constexpr int kQBlock = kPtRows * 128;
  static constexpr int kQTile = (kQ8 ? 2 : kDB) * kQBlock;
  static constexpr int kGroup = kDB * 1024;          // a K or V tile's 8-row group: [column block][8][128 bytes]
  static constexpr int kTileBytes = kPtKeys / 8 * kGroup;
  // kQ8: K tiles of 128-byte rows, V tiles of codes as [8 rows][column block][8][64 bytes]
  static constexpr int kKTile = kQ8 ? kPtKeys * 128 : kTileBytes;
  static constexpr int kVTile = kQ8 ? kTileBytes / 2 : kTileBytes;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + 2 * kQTile;
  static constexpr int kOffV = kOffK + kPtSlots * kKTile;
  static constexpr int kOffVb = kOffV + kPtSlots * kVTile;
  static constexpr int kOffPar = kOffVb + (kQ8 ? kPtVbSlots * kTileBytes : 0);
  // kQ8: scales, and those of a piece's rows.  Blocks of 16 rows or more: four rounds of 8 tiles, of each four of
  // K's and four of V's exponents e, and whether one of those is far (q8_far); shorter ones: a tile in each ring slot,
  // {K's, e, 2^-e} of every key, no number for the last where e is far
  static constexpr int kOffScale = kOffPar + kMaxNodes * 4;
  static constexpr int kScaleBytes = !kQ8 ? 0 : kQ == kPtQ8Fine ? kPtSlots * kPtKeys * 12 : 4 * kPtRound * 4;
  static constexpr int kOffBar = kOffScale + kScaleBytes + (kQ8 ? 2 * kPtRows * 4 : 0);
  static constexpr int kSmemAlloc = kOffBar + 640 + 1024;  // slack for 1024-byte alignment
  static constexpr uint32_t kColO = 256;
  static_assert(kSmemAlloc + 8192 <= 232448, "shared memory per CTA");  // 8192: paged_span's and the pieces'
};

struct PtBars {
  uint64_t q_full[2];
  uint64_t k_full[kPtSlots];
  uint64_t k_empty[kPtSlots];
  uint64_t v_full[kPtSlots];
  uint64_t v_empty[kPtSlots];
  uint64_t s_full[2][2];
  uint64_t p_full[2][2];
  uint64_t pv_done[2][2];
  uint64_t o_done;
  uint64_t s_done[2];
  uint64_t o_free[2];  // tile x's warps have read O
  uint64_t rows_met;   // the softmax warps meet
  uint64_t vb_full[kPtVbSlots];   // kQ8: V tiles as fp16
  uint64_t vb_empty[kPtVbSlots];
  uint64_t scale_full[kPtSlots];  // the keys' scales: a tile's, or a round's
  uint64_t rows_read[2];          // tile x's warps have read their rows' scales
  uint64_t piece_full[kPtPieces];
  uint64_t piece_empty[kPtPieces];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(PtBars) <= 640);

// One piece of work, a range of a unit's key tiles: what the producer finds and every warp goes by.
struct PtPiece {
  int b, hk, rt, P, n;  // unit; the sequence's committed and new rows
  int t0, t1;           // of the unit's tiles, those to take
  int c0, c1;           // CTAs that share the unit, c1 <= c0: it is this CTA's alone
  int slot0;            // where CTA c0 parks its part (the others: 2 c)
  int slot;             // and this one
  int more;             // 0: there is none
};
struct PtArgs {
  int NT;      // nodes per row tile
  int tiles;   // row tiles per unit: 2, or 1 (cluster schedule of few tiles)
  int MP;      // units per (sequence, KV head)
  int splits;  // cluster schedule: parts of a pair's keys
  int wide;    // K and V boxes span both column blocks (5-D maps)
};

__device__ __forceinline__ float pt_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float pt_max64(const float (&sv)[64]) {
  float c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) c[k] = fmaxf(sv[2 * k], sv[2 * k + 1]);
#pragma unroll
  for (int j = 8; j < 64; j += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = pt_max3(c[k], sv[j + 2 * k], sv[j + 2 * k + 1]);
  return fmaxf(fmaxf(c[0], c[1]), fmaxf(c[2], c[3]));
}
// P = 2^(s c - m) as bf16 pairs; returns the sum of the unrounded values.  m = -inf: no key
// has been visible yet and every s is -inf, so P is 0 with any finite offset.
__device__ __forceinline__ float pt_exp64(const float (&sv)[64], float c, float m, uint32_t (&pw)[32]) {
  const float nm = m == -INFINITY ? 0.f : -m;
  const float2 cc = make_float2(c, c), nm2 = make_float2(nm, nm);
  float2 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const float2 t = __ffma2_rn(make_float2(sv[2 * k], sv[2 * k + 1]), cc, nm2);
    const float e0 = ptx::ex2(t.x), e1 = ptx::ex2(t.y);
    acc[k & 3] = __fadd2_rn(acc[k & 3], make_float2(e0, e1));
    pw[k] = ptx::cvt_bf16x2(e0, e1);
  }
  const float2 s2 = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
  return s2.x + s2.y;
}
// v[x] of two by selection: a runtime index would put them in local memory, which every step's
// waits would then read again (0.1 us a step)
template <typename T>
__device__ __forceinline__ T pt_of(const T (&v)[2], int x) {
  return x ? v[1] : v[0];
}
// bits [lo, hi) of a 64-bit word
__device__ __forceinline__ uint64_t pt_bits(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 64);
  if (hi <= lo) return 0ull;
  const uint64_t up = hi == 64 ? ~0ull : (1ull << hi) - 1ull;
  return up & ~((1ull << lo) - 1ull);
}

// S of one row tile (K = D in steps of 16) as one asm block: an issuing thread shares its
// sub-partition with softmax warps, and fewer instructions per product issue the short
// (N = 64) products sooner.  bd steps 32 bytes inside a 128-byte row, 1 KB to the second
// column block.
__device__ __forceinline__ void pt_s_product(uint32_t d, const uint64_t (&ad)[8], uint64_t bd, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b32 z;\n\tmov.b32 z, 0;\n\tsetp.ne.b32 p0, z, 0;\n\tsetp.eq.b32 p1, z, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %9, %17, p0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %10, %17, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %11, %17, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %12, %17, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %5, %13, %17, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %6, %14, %17, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %7, %15, %17, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %8, %16, %17, p1;\n\t}" ::"r"(d),
      "l"(ad[0]), "l"(ad[1]), "l"(ad[2]), "l"(ad[3]), "l"(ad[4]), "l"(ad[5]), "l"(ad[6]), "l"(ad[7]), "l"(bd),
      "l"(bd + 2), "l"(bd + 4), "l"(bd + 6), "l"(bd + 64), "l"(bd + 66), "l"(bd + 68), "l"(bd + 70), "r"(idesc)
      : "memory");
}
__device__ __forceinline__ void pt_s_product(uint32_t d, const uint64_t (&ad)[4], uint64_t bd, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) ptx::mma_bf16_ss(d, ad[kk], bd + kk * 2, idesc, kk > 0 ? 1u : 0u);
}
// O += P V of 64 keys: P from TMEM (8 columns per 16 keys), V rows 16 apart (`step` 16-byte units)
__device__ __forceinline__ void pt_pv_product(uint32_t d, uint32_t p, uint64_t vd, uint32_t step, uint32_t idesc,
                                              uint32_t acc0) {
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b32 z;\n\tmov.b32 z, 0;\n\tsetp.ne.b32 p0, %10, 0;\n\tsetp.eq.b32 p1, z, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %5, %9, p0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %6, %9, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %7, %9, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], %8, %9, p1;\n\t}" ::"r"(d),
      "r"(p), "r"(p + 8), "r"(p + 16), "r"(p + 24), "l"(vd), "l"(vd + step), "l"(vd + 2 * step), "l"(vd + 3 * step),
      "r"(idesc), "r"(acc0)
      : "memory");
}

// kQ8: S of one row tile in e4m3: both parts of Q (16 KB apart) against the same K, 32 columns a step.  One asm
// block at 128 columns, as above
__device__ __forceinline__ void pt_s_product_q8(uint32_t d, uint64_t qd, uint64_t kd, int steps, uint32_t idesc) {
  constexpr uint64_t kPart = kPtRows * 128 / 16;
  if (steps == 4) {
    asm volatile(
        "{\n\t.reg .pred p0, p1;\n\t.reg .b32 z;\n\tmov.b32 z, 0;\n\tsetp.ne.b32 p0, z, 0;\n\tsetp.eq.b32 p1, z, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %9, %13, p0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %2, %10, %13, p1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %3, %11, %13, p1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %4, %12, %13, p1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %5, %9, %13, p1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %6, %10, %13, p1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %7, %11, %13, p1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %8, %12, %13, p1;\n\t}" ::"r"(d),
        "l"(qd), "l"(qd + 2), "l"(qd + 4), "l"(qd + 6), "l"(qd + kPart), "l"(qd + kPart + 2), "l"(qd + kPart + 4),
        "l"(qd + kPart + 6), "l"(kd), "l"(kd + 2), "l"(kd + 4), "l"(kd + 6), "r"(idesc)
        : "memory");
    return;
  }
#pragma unroll 1
  for (int i = 0; i < 2 * steps; ++i) {
    const int kk = i < steps ? i : i - steps;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(qd + (i < steps ? 0 : kPart) + kk * 2), "l"(kd + kk * 2), "r"(idesc), "r"(i > 0 ? 1u : 0u)
        : "memory");
  }
}
__device__ __forceinline__ uint32_t pt_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
constexpr float kPtShift = 7.f;  // P is held times 2^7
// kQ8: P = 2^(s c + e - m) as fp16 pairs, c and e of 16 keys each.  Returns the sum of P's, and in lsum that of
// 2^-e P's
__device__ __forceinline__ float pt_exp64_q8(const float (&sv)[64], const float (&gf)[4], const float (&ge)[4], float m,
                                             uint32_t (&pw)[32], float& lsum) {
  const float nm = m == -INFINITY ? 0.f : kPtShift - m;
  float psum = 0.f;
  lsum = 0.f;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float2 cc = make_float2(gf[g], gf[g]), add = make_float2(ge[g] + nm, ge[g] + nm);
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int k = 8 * g; k < 8 * g + 8; ++k) {
      const float2 t = __ffma2_rn(make_float2(sv[2 * k], sv[2 * k + 1]), cc, add);
      const float e0 = ptx::ex2(t.x), e1 = ptx::ex2(t.y);
      acc[k & 1] = __fadd2_rn(acc[k & 1], make_float2(e0, e1));
      pw[k] = pt_f16x2(e0, e1);
    }
    const float2 both = __fadd2_rn(acc[0], acc[1]);
    const float all = both.x + both.y;
    psum += all;
    lsum = fmaf(all, ptx::ex2(-ge[g]), lsum);
  }
  return psum;
}
__device__ __forceinline__ float pt_max64_q8(const float (&sv)[64], const float (&gf)[4], const float (&ge)[4]) {
  float m = -INFINITY;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float x = pt_max3(sv[16 * g], sv[16 * g + 1], sv[16 * g + 2]);
#pragma unroll
    for (int j = 3; j < 15; j += 2) x = pt_max3(x, sv[16 * g + j], sv[16 * g + j + 1]);
    m = fmaxf(m, fmaf(fmaxf(x, sv[16 * g + 15]), gf[g], ge[g]));
  }
  return m;
}
// The same with a factor of every key, which is in sv already, and its e and 2^-e (sc[kPtKeys ..] and
// sc[2 kPtKeys ..]).  They are read where they are used, 16 keys' at a time: 64 do not fit the registers.
__device__ __forceinline__ float pt_exp64_fine(const float (&sv)[64], float c, const float* sc, float m,
                                               uint32_t (&pw)[32], float& lsum) {
  const float nm = m == -INFINITY ? 0.f : kPtShift - m;
  float psum = 0.f;
  lsum = 0.f;
#pragma unroll
  for (int j = 0; j < 64; j += 4) {
    const float4 e = *reinterpret_cast<const float4*>(sc + kPtKeys + j);
    const float4 f = *reinterpret_cast<const float4*>(sc + 2 * kPtKeys + j);
    const float e0 = ptx::ex2(fmaf(sv[j], c, e.x + nm)), e1 = ptx::ex2(fmaf(sv[j + 1], c, e.y + nm));
    const float e2 = ptx::ex2(fmaf(sv[j + 2], c, e.z + nm)), e3 = ptx::ex2(fmaf(sv[j + 3], c, e.w + nm));
    psum += (e0 + e1) + (e2 + e3);
    lsum = fmaf(e0, f.x, fmaf(e1, f.y, fmaf(e2, f.z, fmaf(e3, f.w, lsum))));
    pw[j / 2] = pt_f16x2(e0, e1);
    pw[j / 2 + 1] = pt_f16x2(e2, e3);
    if (j % 16 == 12) asm volatile("" ::: "memory");
  }
  return psum;
}
__device__ __forceinline__ float pt_max64_fine(const float (&sv)[64], float c, const float* sc) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < 64; j += 4) {
    const float4 e = *reinterpret_cast<const float4*>(sc + kPtKeys + j);
    m = fmaxf(fmaxf(m, fmaf(sv[j], c, e.x)), fmaf(sv[j + 1], c, e.y));
    m = fmaxf(fmaxf(m, fmaf(sv[j + 2], c, e.z)), fmaf(sv[j + 3], c, e.w));
    if (j % 16 == 12) asm volatile("" ::: "memory");
  }
  return m;
}

// y 2^x += l 2^ref, l >= 0 or NaN
__device__ __forceinline__ void pt_add(float& y, float& x, float l, float ref) {
  const float top = fmaxf(x, ref), base = top == -INFINITY ? 0.f : top;
  y = y * ptx::ex2(x - base) + l * ptx::ex2(ref - base);
  x = top;
}

// Wait for this piece's own copies or products even when another wait has run out.
__device__ __forceinline__ void pt_drain(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  int quiet = 0;
  if (!ptx::mbar_wait(bar, parity, &quiet)) *abort_flag = 1;
}

// Bounded waits in few lines (kShort): the roles' loops share the instruction caches, and what one of them takes more,
// the softmax warps wait for (misses a step 77, of the bf16 kernel 18).  kNap: a role that runs ahead of
// the others sleeps between looks.  Gives up after kPtLooks looks, some seconds, or when another has.
constexpr uint32_t kPtLooks = 1u << 26;
template <bool kNap>
__device__ __forceinline__ bool pt_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (uint32_t n = 0; !ptx::mbar_try_wait(bar, parity);) {
    if (kNap) __nanosleep(64);
    n += kNap ? 16 : 1;
    if (__builtin_expect((n & 1023u) == 0, 0) && (*abort || n >= kPtLooks)) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
template <bool kShort>
__device__ __forceinline__ bool pt_wait_for(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if constexpr (kShort) return pt_wait<false>(bar, parity, abort);
  return ptx::mbar_wait(bar, parity, abort);
}

__device__ __forceinline__ void pt_bars_init(PtBars* bars, bool q8, bool fine, int warps) {
  ptx::mbar_init(&bars->q_full[0], q8 ? 4 : 1);  // converter warps, or the copies
  ptx::mbar_init(&bars->q_full[1], q8 ? 4 : 1);
  ptx::mbar_init(&bars->rows_met, 8);
  for (int s = 0; s < kPtVbSlots; ++s) {
    ptx::mbar_init(&bars->vb_full[s], 4);
    ptx::mbar_init(&bars->vb_empty[s], 1);
  }
  for (int s = 0; s < kPtSlots; ++s) ptx::mbar_init(&bars->scale_full[s], fine ? 4 : 1);
  ptx::mbar_init(&bars->rows_read[0], 4);
  ptx::mbar_init(&bars->rows_read[1], 4);
  for (int s = 0; s < kPtPieces; ++s) {
    ptx::mbar_init(&bars->piece_full[s], 1);
    ptx::mbar_init(&bars->piece_empty[s], warps - 1);
  }
  for (int s = 0; s < kPtSlots; ++s) {
    ptx::mbar_init(&bars->k_full[s], 1);
    ptx::mbar_init(&bars->k_empty[s], q8 ? 6 : 2);  // both S issuers (q8: K and V share a barrier; the converters)
    ptx::mbar_init(&bars->v_full[s], 1);
    ptx::mbar_init(&bars->v_empty[s], 1);
  }
  for (int x = 0; x < 2; ++x)
    for (int u = 0; u < 2; ++u) {
      ptx::mbar_init(&bars->s_full[x][u], 1);
      ptx::mbar_init(&bars->p_full[x][u], 4);
      ptx::mbar_init(&bars->pv_done[x][u], 1);
    }
  ptx::mbar_init(&bars->o_done, 1);
  ptx::mbar_init(&bars->s_done[0], 1);
  ptx::mbar_init(&bars->s_done[1], 1);
  ptx::mbar_init(&bars->o_free[0], 4);
  ptx::mbar_init(&bars->o_free[1], 4);
  ptx::fence_mbar_init();
}

template <int D, int kCap, bool kStream, int kQ>
__global__ void __launch_bounds__(PtCfg<D, kQ>::kThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, PagedAttn a, PtArgs pa) {
  ptx::griddep_launch_dependents();
  using C = PtCfg<D, kQ>;
  constexpr bool kQ8 = C::kQ8, kFine = kQ == kPtQ8Fine;
  // capped scores over bf16 pages too: two chunks of 2048 rows over 3000 to 4000 took 474 us with the longer waits, now
  // 360; without a cap those are 1 to 2 % faster
  constexpr bool kShort = kQ8 || kCap != kNoCap;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t mis = ptx::smem_addr(smem_raw) & 1023u;
  unsigned char* sm = smem_raw + ((1024u - mis) & 1023u);
  unsigned char* sQ = sm + C::kOffQ;
  unsigned char* sK = sm + C::kOffK;
  unsigned char* sV = sm + C::kOffV;
  int* s_par = reinterpret_cast<int*>(sm + C::kOffPar);
  PtBars* bars = reinterpret_cast<PtBars*>(sm + C::kOffBar);
  volatile int* abort_flag = &bars->abort;
  __shared__ unsigned long long s_red[kPagedRed];
  __shared__ int s_last;
  __shared__ PtPiece s_piece[kPtPieces];

  // warp: the role, in the order of the bf16 kernel's warps (12..15: converters)
  const int hw_warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warp = !kQ8 || hw_warp >= 12 ? hw_warp : hw_warp < 2 ? hw_warp : hw_warp < 4 ? hw_warp + 8 : hw_warp - 2;
  float* s_scale = reinterpret_cast<float*>(sm + C::kOffScale);
  float* s_rscale = reinterpret_cast<float*>(sm + C::kOffScale + C::kScaleBytes);
  const int NT = pa.NT, rows_used = a.G * NT, RT = pa.tiles * rows_used;
  if (warp == 1) {
    ptx::tmem_alloc(&bars->tmem_base, 512);
    ptx::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&tmQ);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
    bars->abort = 0;
    pt_bars_init(bars, kQ8, kFine, C::kThreads / 32);
  }
  // the Q rows that no box fills
  for (int r = rows_used + threadIdx.x; !kQ8 && r < 2 * kPtRows; r += C::kThreads) {
    const int x = r >= kPtRows ? 1 : 0, rr = r - x * kPtRows;
    if (rr < rows_used) continue;
    for (int db = 0; db < C::kDB; ++db) {
      uint4* row = reinterpret_cast<uint4*>(sQ + x * C::kQTile + db * C::kQBlock + rr * 128);
#pragma unroll
      for (int k = 0; k < 8; ++k) row[k] = make_uint4(0, 0, 0, 0);
    }
  }
  ptx::fence_proxy_async_smem();
  // shared memory, TMEM and parameters only so far: this overlaps the previous kernel's tail
  ptx::griddep_wait();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // ---- this CTA's pieces
  UnitWalk w{};  // the producer's
  const size_t cta = ((size_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;  // cluster schedule
  if constexpr (kStream) {
    const PagedSpan sp = paged_span<true>(a, RT, kPtKeys, 1, s_red, kPtTol, kPtFix);
    w = unit_walk(sp);
  }
  // the pieces, by the softmax warps, by the others, or by all (bf16): a warp's registers are fixed from
  // setmaxnreg on, so with 8-bit pages the two have code of their own
  enum { kAll, kSoftmax, kOthers };
  auto run_pieces = [&](auto who) {
  constexpr int kWho = decltype(who)::value;
  // the softmax warps meet.  Between pieces by an mbarrier: a hardware barrier would hang if the wait for a
  // piece ran out in some of them only
  unsigned met = 0;
  auto softmax_sync = [&] {
    if constexpr (kStream) {
      int quiet = 0;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars->rows_met);
      if (!ptx::mbar_wait(&bars->rows_met, met & 1, &quiet)) *abort_flag = 1;
      ++met;
      __syncwarp();
    } else {
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
  };
  int loaded_b = -1, n_act = 0;
  // tiles, and tiles with rows of A and B, of the pieces before this one, and how many those were: what
  // the rings' slots and the barriers' phases go by.  Every role counts them alike.
  unsigned kt = 0, done_x[2] = {0, 0}, pieces = 0, rounds = 0;  // rounds: of 8 tiles
  unsigned k_issued = 0, v_issued = 0;  // the producer's copies
  unsigned q_loads = 0;                 // an S issuer's
  bool ok = true;                       // no wait of this role has run out
  auto drain = [&] {  // the producer: no copy is in flight when the CTA ends
    for (unsigned s = 0; s < kPtSlots; ++s) {
      if (s < k_issued) pt_drain(&bars->k_full[s], ((k_issued - 1 - s) / kPtSlots) & 1, abort_flag);
      if (s < v_issued) pt_drain(&bars->v_full[s], ((v_issued - 1 - s) / kPtSlots) & 1, abort_flag);
    }
  };
  for (unsigned np = 0;; ++np) {
    PtPiece pc;
    if constexpr (kStream) {
      // the producer runs ahead of the others: it finds the pieces and posts them
      const int ps = np % kPtPieces;
      int quiet = 0;  // pieces come after an abort too, so that each cut unit's parts are counted
      if (kWho != kSoftmax && warp == 0) {
        pc.more = unit_next(a, w, RT, kPtKeys);
        pc.b = w.b, pc.hk = w.hk, pc.rt = w.rt, pc.P = w.P, pc.n = w.n, pc.t0 = w.t0, pc.t1 = w.t1;
        const UnitCtas by = unit_ctas(w);
        pc.c0 = (int)by.c0, pc.c1 = (int)by.c1;
        pc.slot0 = unit_slot(by.c0, w.per, w.u0), pc.slot = unit_slot(blockIdx.x, w.per, w.u0);
        bool got = true;
        if (np >= kPtPieces)
          got = ptx::mbar_wait_limit(&bars->piece_empty[ps], (np / kPtPieces - 1) & 1, &quiet, 8 * TV_WAIT_NS);
        if (!__all_sync(0xffffffffu, got)) {
          *abort_flag = 1;
          break;
        }
        if (lane == 0) {
          s_piece[ps] = pc;
          ptx::mbar_arrive(&bars->piece_full[ps]);
        }
        __syncwarp();
      } else {
        const bool got =
            ptx::mbar_wait_limit(&bars->piece_full[ps], (np / kPtPieces) & 1, &quiet, 8 * TV_WAIT_NS);
        if (!__all_sync(0xffffffffu, got)) {
          *abort_flag = 1;
          break;
        }
        const PtPiece& at = s_piece[ps];
        pc.b = at.b, pc.hk = at.hk, pc.rt = at.rt, pc.P = at.P, pc.n = at.n, pc.t0 = at.t0, pc.t1 = at.t1;
        pc.more = at.more;
      }
      if (!pc.more) break;
    } else {
      pc.b = blockIdx.z, pc.hk = blockIdx.y, pc.rt = pa.MP - 1 - (int)blockIdx.x / pa.splits;
    }
    const int b = pc.b, hk = pc.hk, mp = pc.rt;
    if (b != loaded_b) {
      // Tree rows count up to the first padding row (a tree with rows behind it is bad).  Every warp
      // counts for itself, and the softmax warps check and keep the parents.  The first reads
      // run beside those of the lengths.
      const int32_t* par = a.parent ? a.parent + (size_t)b * a.N : nullptr;
      const int st = (warp - 2) * 32 + lane;
      const bool rows_warp = kWho != kOthers && warp >= 2 && warp < 10;
      int first[4], p_first = -1, p_before = -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) first[k] = par && k * 32 + lane < a.N ? par[k * 32 + lane] : -1;
      if (par && rows_warp && st < a.N) {
        p_first = par[st];
        if (st > 0) p_before = par[st - 1];
      }
      if constexpr (!kStream) {
        bool bad = false;
        pc.P = a.prefix_len[b];
        pc.n = paged_rows(a, b, pc.P, &bad);
        if (pc.n == 0) pc.P = 0;
        if (threadIdx.x == 0 && (bad || paged_cut(a, b, pc.P, pc.n))) set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
      }
      const int n = pc.n;
      n_act = n;
      if (par && n > 0) {
        int count = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = k * 32 + lane;
          count += t > 0 && t < n && first[k] != -1;
        }
        for (int t = 128 + lane; t < n; t += 32) count += par[t] != -1;
        n_act = 1 + __reduce_add_sync(0xffffffffu, count);
        if (rows_warp) {
          if (loaded_b >= 0) softmax_sync();  // the piece before's rows have read s_par
          for (int t = st; t < n; t += 256) {
            const int p = t == st ? p_first : par[t];
            const bool prev_pad = t >= 2 && (t == st ? p_before : par[t - 1]) == -1;
            const bool fits = t == 0 ? p == -1 : (p == -1 || (p >= 0 && p < t && !prev_pad));
            if (!fits) set_dev_status(a.dev_status, TV_DEV_BAD_TREE);
            s_par[t] = fits ? p : -1;
          }
          softmax_sync();
        }
      }
      loaded_b = b;
    }
    const int P = pc.P, n = pc.n;
    const int lo = unit_lo(a, P, mp, RT);
    int split = 0;
    if constexpr (!kStream) {
      const int T_u = unit_tiles(a, P, n, mp, RT, kPtKeys);
      split = blockIdx.x % pa.splits;
      pc.t0 = (int)((long long)T_u * split / pa.splits);
      pc.t1 = (int)((long long)T_u * (split + 1) / pa.splits);
    }
    const int t_begin = lo / kPtKeys + pc.t0;  // this piece's key tiles
    const int nt_all = pc.t1 - pc.t0;
    const int key_end = P + n_act;  // rows from here on, and before lo, may hold anything
    int i0[2], ntx[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      i0[x] = (pa.tiles * mp + x) * NT;
      const int hi = x < pa.tiles && i0[x] < n_act ? P + min(n_act, i0[x] + NT) : 0;
      ntx[x] = max(0, min(nt_all, (hi + kPtKeys - 1) / kPtKeys - t_begin));
    }
    const int nt = max(ntx[0], ntx[1]);

    float m_run = -INFINITY, l_run = 0.f;
    bool have_o = false;
    // kQ8: the weights of tiles with a far scale (q8_far; now), from one with a large scale on of all (high), add up to
    // l_far times 2^z_ref
    float l_far = 0.f, z_ref = -INFINITY;
    bool now = false, high = false;
    if (kWho != kSoftmax && warp == 0) {
      // ---------------------------------------------------------------- producer
      // lane: row piece pi of a tile (and, without 5-D boxes, its column block db)
      const int per_piece = pa.wide ? 1 : C::kDB;
      const int box_shift = min(a.page_shift, C::kDB == 1 || pa.wide ? 6 : 3);
      const int db = lane % per_piece, pi = lane / per_piece;
      const bool in_tile = (pi << box_shift) < kPtKeys;
      const uint32_t box_bytes = (uint32_t)((kQ8 ? 64 : 128) * C::kDB / per_piece) << box_shift;  // kQ8: of V
      const int32_t* table = a.table + (size_t)b * a.max_pages;
      // whether this lane's box in tile t holds a needed row, and its table entry (read two tiles
      // ahead, checked when it is used)
      auto needed = [&](int t) -> bool {
        const int j = (t_begin + t) * kPtKeys + (pi << box_shift);
        return t < nt && in_tile && j < key_end && j + (1 << box_shift) > lo;
      };
      auto entry = [&](int t) -> int {
        return needed(t) ? table[((t_begin + t) * kPtKeys + (pi << box_shift)) >> a.page_shift] : 0;
      };
      auto checked = [&](int t, int page) -> int {
        if (!needed(t)) return -1;
        if (page >= 0 && page < a.num_pages) return page;
        set_dev_status(a.dev_status, TV_DEV_BAD_PAGE);
        return -1;
      };
      int raw0 = entry(0), raw1 = entry(1), before = -1;
      if constexpr (kQ8) {
        // K and V of a tile come together: a K box holds whole 128-byte rows, column blocks or not
#pragma unroll 1
        for (int t = 0; t < nt; ++t) {
          const int page = checked(t, raw0);
          raw0 = raw1;
          raw1 = entry(t + 2);
          const unsigned gt = kt + t;
          const int slot = gt % kPtSlots;
          bool got = true;
          if (gt >= kPtSlots) got = pt_wait<true>(&bars->k_empty[slot], ((gt / kPtSlots) - 1) & 1, abort_flag);
          if (!(ok = __all_sync(0xffffffffu, got))) break;
          const uint32_t v_boxes = __popc(__ballot_sync(0xffffffffu, page >= 0));
          const uint32_t k_boxes = __popc(__ballot_sync(0xffffffffu, page >= 0 && db == 0));
          if (lane == 0)
            ptx::mbar_arrive_expect_tx(&bars->k_full[slot], v_boxes * box_bytes + (k_boxes * 128u << box_shift));
          __syncwarp();
          if (page >= 0) {
            const int row = ((t_begin + t) * kPtKeys + (pi << box_shift)) & ((1 << a.page_shift) - 1);
            const int group = (pi << box_shift) >> 3, plane = page * a.Hkv + hk;
            unsigned char* to_v = sV + slot * C::kVTile + group * (C::kGroup / 2) + db * 512;
            if (db == 0)
              ptx::tma_load_3d(sK + slot * C::kKTile + group * 1024, &tmK, &bars->k_full[slot], 0, row, plane);
            if (C::kDB > 1 && pa.wide)
              ptx::tma_load_5d(to_v, &tmV, &bars->k_full[slot], 0, 0, 0, row >> 3, plane);
            else
              ptx::tma_load_3d(to_v, &tmV, &bars->k_full[slot], db * 64, row, plane);
          }
          __syncwarp();
          k_issued = gt + 1;
        }
      } else {
        // this lane's box of tile t into its ring slot; false after an abort
        auto fetch = [&](unsigned char* ring, const CUtensorMap* tm, uint64_t* full, uint64_t* empty, int t,
                         int pg) -> bool {
          const unsigned gt = kt + t;
          const int slot = gt % kPtSlots;
          bool got = true;
          if (gt >= kPtSlots) got = pt_wait_for<kShort>(&empty[slot], ((gt / kPtSlots) - 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, got)) return false;
          const uint32_t boxes = __ballot_sync(0xffffffffu, pg >= 0);
          if (lane == 0) ptx::mbar_arrive_expect_tx(&full[slot], __popc(boxes) * box_bytes);
          __syncwarp();
          if (pg >= 0) {
            const int row = ((t_begin + t) * kPtKeys + (pi << box_shift)) & ((1 << a.page_shift) - 1);
            unsigned char* dst = ring + slot * C::kTileBytes + ((pi << box_shift) >> 3) * C::kGroup + db * 1024;
            if (C::kDB > 1 && pa.wide)
              ptx::tma_load_5d(dst, tm, &full[slot], 0, 0, 0, row >> 3, pg * a.Hkv + hk);
            else
              ptx::tma_load_3d(dst, tm, &full[slot], db * 64, row, pg * a.Hkv + hk);
          }
          return true;
        };
        for (int t = 0; ok && t <= nt && nt > 0; ++t) {
          const int page = checked(t, raw0);
          raw0 = raw1;
          raw1 = entry(t + 2);
          if (t < nt) {
            if (!(ok = fetch(sK, &tmK, bars->k_full, bars->k_empty, t, page))) break;
            k_issued = kt + t + 1;
          }
          if (t > 0) {
            if (!(ok = fetch(sV, &tmV, bars->v_full, bars->v_empty, t - 1, before))) break;
            v_issued = kt + t;
          }
          before = page;
        }
      }
      if (!kStream && lane == 0) drain();
    } else if (kWho != kSoftmax && (warp == 1 || warp == 11)) {
      // ---------------------------------------------------------------- S issuer of tile x
      const int x = warp == 1 ? 0 : 1;
      if (lane == 0) {
        const int ntm = pt_of(ntx, x);
        const unsigned dx = pt_of(done_x, x);
        if constexpr (kQ8) {
          // also where the tile has no rows: the converters go by s_done, which may not run ahead of them
          if (nt > 0) ok = ok && pt_wait_for<kShort>(&bars->q_full[x], pieces & 1, abort_flag);
        } else if (ntm > 0) {
          ptx::mbar_arrive_expect_tx(&bars->q_full[x], (uint32_t)(rows_used * 128 * C::kDB));
          for (int g = 0; g < a.G; ++g)
            for (int d = 0; d < C::kDB; ++d)
              ptx::tma_load_3d(sQ + x * C::kQTile + d * C::kQBlock + g * NT * 128, &tmQ, &bars->q_full[x], d * 64,
                               pt_of(i0, x), b * a.Hq + hk * a.G + g);
          pt_drain(&bars->q_full[x], q_loads++ & 1, abort_flag);
        }
        if (nt > 0) {
          constexpr uint32_t idS = ptx::idesc_bf16(kPtRows, kPtKeys, false, false);
          const uint32_t qaddr = ptx::smem_addr(sQ + x * C::kQTile);
          uint64_t adq[D / 16];
#pragma unroll
          for (int kk = 0; kk < (kQ8 ? 1 : D / 16); ++kk)
            adq[kk] = ptx::sdesc_sw128(qaddr + (kk >> 2) * C::kQBlock + (kk & 3) * 32, 16, 1024);
          for (int t = 0; ok && t < nt; ++t) {
            const int ks = (kt + t) % kPtSlots;
            if (!(ok = pt_wait_for<kShort>(&bars->k_full[ks], ((kt + t) / kPtSlots) & 1, abort_flag))) break;
            if (t < ntm) {
              // S_X(t) overwrites P_X of two tiles before in this buffer
              const unsigned tx = dx + t;
              const int buf = tx & 1;
              if (tx >= 2 && !(ok = pt_wait_for<kShort>(&bars->pv_done[x][buf], ((tx - 2) >> 1) & 1, abort_flag))) break;
              ptx::tc_fence_after();
              if constexpr (kQ8)
                pt_s_product_q8(tmem + x * kPtRows + buf * kPtKeys, adq[0],
                                ptx::sdesc_sw128(ptx::smem_addr(sK + ks * C::kKTile), 16, 1024), a.D / 32,
                                idS & ~(7u << 7 | 7u << 10));  // e4m3 operands
              else
                pt_s_product(tmem + x * kPtRows + buf * kPtKeys, adq,
                             ptx::sdesc_sw128(ptx::smem_addr(sK + ks * C::kTileBytes), 16, C::kGroup), idS);
              ptx::mma_commit(&bars->s_full[x][buf]);
            }
            ptx::mma_commit(&bars->k_empty[ks]);
          }
          // Q's place is free again behind its products
          ptx::mma_commit(&bars->s_done[x]);
          pt_drain(&bars->s_done[x], pieces & 1, abort_flag);
        }
      }
      __syncwarp();
    } else if (kWho != kSoftmax && warp == 10) {
      // ---------------------------------------------------------------- PV issuer
      // kQ8: fp16 operands
      constexpr uint32_t idO = ptx::idesc_bf16(kPtRows, D, false, true) & (kQ8 ? ~(7u << 7 | 7u << 10) : ~0u);
      // only the first and last tile can hold V rows that may be anything; the warp zeroes them
      // (their weights are zero too) before its lane 0 issues that tile.  A loop that kept all
      // lanes together for every tile cost 3 %
      auto edge = [&](int t) -> bool {
        const int j0 = (t_begin + t) * kPtKeys;
        return !kQ8 && t >= 0 && t < nt && (j0 < lo || j0 + kPtKeys > key_end);  // kQ8: the converters do that
      };
      auto zero_rows = [&](int t) {
        const int vs = (kt + t) % kPtSlots, j0 = (t_begin + t) * kPtKeys;
        if (!pt_wait_for<kShort>(&bars->v_full[vs], ((kt + t) / kPtSlots) & 1, abort_flag)) return;
        for (int r = lane; r < kPtKeys; r += 32)
          if (j0 + r < lo || j0 + r >= key_end)
            for (int db = 0; db < C::kDB; ++db) {
              uint4* row =
                  reinterpret_cast<uint4*>(sV + vs * C::kTileBytes + (r >> 3) * C::kGroup + db * 1024 + (r & 7) * 128);
#pragma unroll
              for (int k = 0; k < 8; ++k) row[k] = make_uint4(0, 0, 0, 0);
            }
        ptx::fence_proxy_async_smem();
      };
      auto issue = [&](int t) -> bool {
        constexpr int kSlots = kQ8 ? kPtVbSlots : kPtSlots;
        const int vs = (kt + t) % kSlots;
        if (!pt_wait_for<kShort>(kQ8 ? &bars->vb_full[vs] : &bars->v_full[vs], ((kt + t) / kSlots) & 1, abort_flag))
          return false;
        const uint64_t vd =
            ptx::sdesc_sw128(ptx::smem_addr((kQ8 ? sm + C::kOffVb : sV) + vs * C::kTileBytes), 1024, C::kGroup);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (t >= ntx[x]) continue;
          const unsigned tx = done_x[x] + t;
          const int buf = tx & 1;
          if (!pt_wait_for<kShort>(&bars->p_full[x][buf], (tx >> 1) & 1, abort_flag)) return false;
          ptx::tc_fence_after();
          pt_pv_product(tmem + C::kColO + x * kPtRows, tmem + x * kPtRows + buf * kPtKeys, vd, 2 * C::kGroup / 16, idO,
                        t > 0 ? 1u : 0u);  // P: 8 columns per 16 keys
          ptx::mma_commit(&bars->pv_done[x][buf]);
        }
        ptx::mma_commit(kQ8 ? &bars->vb_empty[vs] : &bars->v_empty[vs]);
        return true;
      };
      const int last = nt - 1;
      // one copy of the loop's code: a kernel of few steps pays for each line that it fetches first
#pragma unroll 1
      for (int part = 0, t = 0; part < 2; ++part) {
        const int from = part == 0 ? 0 : last, to = part == 0 ? last : nt;
        if (from < to && edge(from)) zero_rows(from);
        __syncwarp();
        // the piece before's O has been read
        if (kStream && part == 0 && pieces > 0 && nt > 0)
          for (int x = 0; x < 2; ++x)
            ok = __all_sync(0xffffffffu, ok && pt_wait_for<kShort>(&bars->o_free[x], (pieces - 1) & 1, abort_flag));
        if (lane == 0)
          for (; ok && t < to; ++t) ok = issue(t);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      if (lane == 0 && nt > 0) {
        ptx::mma_commit(&bars->o_done);
        pt_drain(&bars->o_done, pieces & 1, abort_flag);
      }
      __syncwarp();
    } else if (kQ8 && kWho == kOthers) {
      // ---------------------------------------------------------------- converters
      const int cw = warp - 12;
      // Q of both tiles as e4m3 parts: eight lanes a row, 16 elements each, four rows a warp at a time
      for (int x = 0; ok && x < 2 && nt > 0; ++x) {
        // the piece before's products have read Q, and its rows their scales
        if (pieces > 0)
          ok = __all_sync(0xffffffffu, pt_wait_for<kShort>(&bars->s_done[x], (pieces - 1) & 1, abort_flag) &&
                                           pt_wait_for<kShort>(&bars->rows_read[x], (pieces - 1) & 1, abort_flag));
        if (!ok) break;
        unsigned char* sQx = sQ + x * C::kQTile;
        const int part = lane & 7;
#pragma unroll 1
        for (int it = 0; it < kPtRows / 16 && pt_of(ntx, x) > 0; it += 2) {
          uint4 v[2][2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int r = (it + u) * 16 + cw * 4 + (lane >> 3), g = r / NT, node = pt_of(i0, x) + r % NT;
            v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
            if (r < rows_used && node < n_act && part * 16 < a.D) {
              const uint4* src = reinterpret_cast<const uint4*>(
                  reinterpret_cast<const uint16_t*>(a.q) +
                  (((size_t)b * a.Hq + hk * a.G + g) * a.N + node) * a.D + part * 16);
              v[u][0] = __ldg(src), v[u][1] = __ldg(src + 1);
            }
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int r = (it + u) * 16 + cw * 4 + (lane >> 3);
            const uint32_t w[8] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w, v[u][1].x, v[u][1].y, v[u][1].z, v[u][1].w};
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) m = __vmaxu2(m, w[k] & 0x7f807f80u);
            int top = (int)(max(m >> 16, m & 0xffffu) >> 7);  // the row's largest exponent field
#pragma unroll
            for (int o = 1; o < 8; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            // below 2^8: elements of the top binade reach 1.99 * 2^7
            const int shift = top == 255 ? 0 : min(127, 134 - max(top, 1));
            const float f = q8_two(shift);
            uint32_t hi[4], lo4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float x0 = __uint_as_float(w[2 * k] << 16) * f, x1 = __uint_as_float(w[2 * k] & 0xffff0000u) * f;
              const float x2 = __uint_as_float(w[2 * k + 1] << 16) * f;
              const float x3 = __uint_as_float(w[2 * k + 1] & 0xffff0000u) * f;
              hi[k] = q8_code4(x0, x1, x2, x3);
              const float4 y = q8_numbers(hi[k], 1.f);
              lo4[k] = q8_code4(x0 - y.x, x1 - y.y, x2 - y.z, x3 - y.w);
            }
            // 128-byte rows, swizzled as the products read them
            unsigned char* to = sQx + r * 128 + ((part ^ (r & 7)) << 4);
            *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(to + C::kQBlock) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
            if (part == 0) s_rscale[x * kPtRows + r] = q8_two(-shift);
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->q_full[x]);
      }
      // Scales.  Blocks of 16 keys or more: warp 12 alone brings those of 8 tiles at once (lane: tile lane / 4, keys
      // 16 (lane % 4)..), looked up a round ahead, their pages two.  Shorter ones: each warp those of its 16
      // keys (lanes 0..15 V's, 16..31 K's), looked up kPtAhead tiles ahead, their pages twice that.
      const int32_t* table = a.table + (size_t)b * a.max_pages;
      auto key_of = [&](int t) -> int {  // this lane's in tile t (or, in rounds, from t on)
        return kFine ? (t_begin + t) * kPtKeys + cw * 16 + (lane & 15)
                     : (t_begin + t + (lane >> 2)) * kPtKeys + (lane & 3) * 16;
      };
      auto page_of = [&](int t) -> int {
        const int j = key_of(t);
        const bool in = kFine ? t < nt : t + (lane >> 2) < nt;
        return in && j + (kFine ? 0 : 15) >= lo && j < key_end ? table[j >> a.page_shift] : -1;
      };
      // K's byte and V's, in bits 8..15, or one of them; 127 where no row needs it
      auto bytes_of = [&](int t, int page) -> int {
        if (page < 0 || page >= a.num_pages) return 127 | 127 << 8;
        const size_t block = (((size_t)page * a.Hkv + hk) << (a.page_shift - a.block_shift)) +
                             ((key_of(t) & ((1 << a.page_shift) - 1)) >> a.block_shift);
        if (kFine) return lane < 16 ? a.vs[block] : a.ks[block];
        return a.ks[block] | a.vs[block] << 8;
      };
      constexpr int kAhead = kFine ? kPtAhead : 1, kStep = kFine ? 1 : 8;
      const bool looks = kFine || cw == 0;
      int pages_to[2 * kAhead], bytes_to[kAhead];
#pragma unroll
      for (int k = 0; k < 2 * kAhead; ++k) pages_to[k] = looks ? page_of(k * kStep) : -1;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) bytes_to[k] = bytes_of(k * kStep, pages_to[k]);
      // the next bytes in line, behind which another step's are looked up, for tile t on
      auto next_bytes = [&](int t) -> int {
        const int bytes = bytes_to[0];
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k) bytes_to[k] = bytes_to[k + 1];
        bytes_to[kAhead - 1] = bytes_of(t + kAhead * kStep, pages_to[kAhead]);
#pragma unroll
        for (int k = kAhead; k + 1 < 2 * kAhead; ++k) pages_to[k] = pages_to[k + 1];
        pages_to[2 * kAhead - 1] = page_of(t + 2 * kAhead * kStep);
        return bytes;
      };
      for (int t = 0; ok && t < nt; ++t) {
        const unsigned gt = kt + t;
        const int vs = gt % kPtSlots, vb = gt % kPtVbSlots;
        bool got = true;
        if (gt >= kPtVbSlots) got = pt_wait<true>(&bars->vb_empty[vb], (gt / kPtVbSlots - 1) & 1, abort_flag);
        if constexpr (kFine) {
          const int bytes = next_bytes(t), ks = __shfl_sync(0xffffffffu, bytes, 16 + (lane & 15));
          if (lane < 16) {
            float* to = s_scale + vs * 3 * kPtKeys + cw * 16 + lane;
            to[0] = q8_scale(ks);
            to[kPtKeys] = (float)(bytes - 127);
            to[2 * kPtKeys] = q8_far(bytes - 127) ? __uint_as_float(0x7fffffffu) : q8_two(127 - bytes);
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bars->scale_full[vs]);
        } else if (cw == 0 && (t == 0 || t % 8 == 4)) {
          // the first round, then each in the middle of the one before.  Its place is that of four rounds before, a
          // tile or more each, of which no tile is later than that whose ring slot has just been seen free
#pragma unroll 1
          for (int r = t == 0 ? 0 : t + 4; r < nt && r <= t + 4; r += 8) {
            const int bytes = next_bytes(r);
            float* of = s_scale + ((rounds + r / 8) & 3) * kPtRound;
            float* to = of + (lane >> 2) * 8 + (lane & 3);
            to[0] = q8_scale(bytes & 255);
            to[4] = (float)((bytes >> 8) - 127);
            const bool far = __any_sync(0xffffffffu, q8_far((bytes >> 8) - 127));
            if (lane == 0) of[64] = far ? 1.f : 0.f;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars->scale_full[(rounds + r / 8) & 3]);
          }
        }
        got = got && pt_wait<true>(&bars->k_full[vs], (gt / kPtSlots) & 1, abort_flag);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) break;
        const int j0 = (t_begin + t) * kPtKeys + cw * 16;
        const unsigned char* from = sV + vs * C::kVTile + cw * C::kGroup + (lane >> 2) * 64 + (lane & 3) * 16;
        unsigned char* to = sm + C::kOffVb + vb * C::kTileBytes + cw * 2 * C::kGroup + (lane >> 2) * 128;
        const int r7 = lane >> 2;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int row = half * 8 + r7, j = j0 + row;
          const bool needed = j >= lo && j < key_end;
#pragma unroll
          for (int blk = 0; blk < C::kDB; ++blk) {
            uint4 c = make_uint4(0, 0, 0, 0);
            if (needed) c = *reinterpret_cast<const uint4*>(from + half * (C::kGroup / 2) + blk * 512);
            uint32_t out[8];
            q8_half4(c.x, out[0], out[1]);
            q8_half4(c.y, out[2], out[3]);
            q8_half4(c.z, out[4], out[5]);
            q8_half4(c.w, out[6], out[7]);
            unsigned char* row_to = to + half * C::kGroup + blk * 1024;
            const int ch = (lane & 3) * 2;
            *reinterpret_cast<uint4*>(row_to + ((ch ^ r7) << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
            *reinterpret_cast<uint4*>(row_to + (((ch + 1) ^ r7) << 4)) = make_uint4(out[4], out[5], out[6], out[7]);
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&bars->vb_full[vb]);
          ptx::mbar_arrive(&bars->k_empty[vs]);
        }
      }
      __syncwarp();
    } else if (kWho != kOthers) {
      // ---------------------------------------------------------------- softmax rows
      const int x = (warp - 2) >> 2;
      const int q4 = hw_warp & 3;
      const int r = q4 * 32 + lane;
      const int g = r / NT, node = pt_of(i0, x) + r % NT;
      const bool valid = x < pa.tiles && r < rows_used && node < n_act;
      const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
      const uint32_t colS = tmem + lane_base + x * kPtRows;
      const uint32_t colO = tmem + lane_base + C::kColO + x * kPtRows;
      const int ntm = pt_of(ntx, x);
      const unsigned dx = pt_of(done_x, x);
      // the row sees [wlo, whi) and, in a tree, its ancestors; rows that are no row see everything
      // (their results go nowhere)
      int wlo = 0, whi = 0x7fffffff;
      if (valid) {
        int depth = node;
        if (a.parent) {
          whi = P;
          if (a.window > 0) {
            depth = 0;
            for (int at = s_par[node]; at >= 0; at = s_par[at]) ++depth;  // parents fall: it ends
          }
        } else {
          whi = P + node + 1;
        }
        if (a.window > 0) wlo = max(0, P + depth - a.window + 1);  // at least 0: wlo - j0 fits an int
      }
      const float c = kCap == kLargeCap ? kLog2e : kCap ? a.cap * kLog2e : a.scale * kLog2e;
      const float ck = kCap == kLargeCap ? 1.f / a.cap : kCap ? 2.f * kLog2e * a.scale / a.cap : 0.f;
      // kQ8: the row's power of two, for all of the piece
      float row_f = 1.f;
      if (kQ8 && nt > 0) {
        ok = ok && __all_sync(0xffffffffu, pt_wait_for<kShort>(&bars->q_full[x], pieces & 1, abort_flag));
        row_f = s_rscale[x * kPtRows + r];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->rows_read[x]);
      }
      for (int t = 0; ok && t < ntm; ++t) {
        const unsigned tx = dx + t;
        const int buf = tx & 1;
        // kQ8: the tile's scales, read before its scores are there: with the products' operands on the way, shared
        // memory takes long to answer
        const float* scales =
            s_scale + (kFine ? (kt + t) % kPtSlots * 3 * kPtKeys : ((rounds + t / 8) & 3) * kPtRound + t % 8 * 8);
        float gf[4], ge[4];
        if constexpr (kQ8) {
          if (kFine || t % 8 == 0) {
            const unsigned n = kFine ? (kt + t) / kPtSlots : (rounds + t / 8) / 4;
            ok = __all_sync(0xffffffffu, pt_wait_for<kShort>(&bars->scale_full[kFine ? (kt + t) % kPtSlots : (rounds + t / 8) & 3],
                                                        n & 1, abort_flag));
            if (!ok) break;
            if (!kFine) now = scales[64] != 0.f;
          }
          if constexpr (!kFine) {
            const float4 ks = *reinterpret_cast<const float4*>(scales), vs = *reinterpret_cast<const float4*>(scales + 4);
            gf[0] = ks.x * row_f, gf[1] = ks.y * row_f, gf[2] = ks.z * row_f, gf[3] = ks.w * row_f;
            ge[0] = vs.x, ge[1] = vs.y, ge[2] = vs.z, ge[3] = vs.w;
          }
        }
        auto scale_keys = [&](float(&v)[64]) {
#pragma unroll
          for (int j = 0; j < 64; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(scales + j);
            v[j] *= f.x * row_f, v[j + 1] *= f.y * row_f, v[j + 2] *= f.z * row_f, v[j + 3] *= f.w * row_f;
            if (j % 16 == 12) asm volatile("" ::: "memory");
          }
        };
        ok = __all_sync(0xffffffffu, pt_wait_for<kShort>(&bars->s_full[x][buf], (tx >> 1) & 1, abort_flag));
        if (!ok) break;
        ptx::tc_fence_after();
        const int j0 = (t_begin + t) * kPtKeys;
        uint64_t vis = ~0ull;
        if (j0 < wlo || j0 + kPtKeys > whi) {
          vis = pt_bits(wlo - j0, whi - j0);
          if (a.parent) {
            int steps = a.window > 0 ? a.window : kMaxNodes + 1;
            for (int at = node; at >= 0 && steps > 0; at = s_par[at], --steps) {
              const int j = P + at - j0;
              if (j < 0) break;  // ancestors only go down from here
              if (j < kPtKeys) vis |= 1ull << j;
            }
          }
        }
        float sv[64];
        auto read_scores = [&] {
          ptx::tmem_ld32(colS + buf * kPtKeys, sv);
          ptx::tmem_ld32(colS + buf * kPtKeys + 32, sv + 32);
          ptx::tmem_wait_ld();
          if constexpr (kFine) scale_keys(sv);
          if constexpr (kCap == kTanhCap) {
            if (vis != ~0ull) {
#pragma unroll
              for (int j = 0; j < 64; ++j)
                if (!((vis >> j) & 1ull)) sv[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 64; j += 4) soft_tanh4(sv + j, kQ == kPtQ8 ? ck * gf[j / 16] : ck);
          } else if constexpr (kCap == kLargeCap) {
            // nearly all scores lie below 0.45 of such a cap; where one does not, the tile is read again
            float z_max = 0.f;
#pragma unroll
            for (int j = 0; j < 64; ++j) {
              const float t = sv[j] * (kQ == kPtQ8 ? a.scale * gf[j / 16] : a.scale), x = t * ck, z = x * x;
              z_max = fmaxf(z_max, z);
              sv[j] = fmaf(t * z, tanh_tail(z), t);
            }
            if (__any_sync(0xffffffffu, z_max >= kTanhNear)) {
              ptx::tmem_ld32(colS + buf * kPtKeys, sv);
              ptx::tmem_ld32(colS + buf * kPtKeys + 32, sv + 32);
              ptx::tmem_wait_ld();
              if constexpr (kFine) scale_keys(sv);
#pragma unroll
              for (int j = 0; j < 64; ++j)
                sv[j] = capped_score(sv[j] * (kQ == kPtQ8 ? a.scale * gf[j / 16] : a.scale), a.cap, ck);
            }
          }
          if (__builtin_expect(vis != ~0ull, 0)) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (!((vis >> j) & 1ull)) sv[j] = -INFINITY;
          }
        };
        if constexpr (!kFine) read_scores();
        // P = 2^(c S - m_run) against a running reference that moves (with a rescale of O) only
        // when a score exceeds it by 2^8: such a score brings the tile's sum to 2^8, so the
        // maximum is taken only then and for the first tile with a visible key
        if constexpr (kQ == kPtQ8) {
          // what the scores are multiplied by; not 0 where one is -inf
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            gf[g] = kCap ? c : gf[g] * c;
            if (vis != ~0ull) gf[g] = fmaxf(gf[g], 1.1754944e-38f);
          }
        }
        auto tile_max = [&]() -> float {
          if constexpr (kFine) return pt_max64_fine(sv, c, scales);
          return pt_max64_q8(sv, gf, ge);
        };
        // The tile's weights by z alone, as P may not hold them.  Scores are read again, eight at a time: these lines sit
        // among those of every tile, and 32 at a time cost tiles without a far scale 3 to 14 %
        auto sum_far = [&](bool mine, float m_before) {
          float large = 0.f;
#pragma unroll 1
          for (int c0 = 0; c0 < kPtKeys; c0 += 8) {
            float z[8], top = z_ref;
            ptx::tmem_ld8(colS + buf * kPtKeys + c0, z);
            ptx::tmem_wait_ld();
            const unsigned seen = (unsigned)(vis >> c0);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              z[j] *= scales[kFine ? c0 + j : c0 / 16] * row_f;
              if constexpr (kCap == kTanhCap) z[j] = soft_tanh(z[j] * ck);
              if constexpr (kCap == kLargeCap) z[j] = capped_score(z[j] * a.scale, a.cap, ck);
              z[j] = seen >> j & 1u ? z[j] * c : -INFINITY;
              top = fmaxf(top, z[j]);
              large = fmaxf(large, scales[kFine ? kPtKeys + c0 + j : 4 + c0 / 16]);
            }
            if (!mine) continue;
            const float base = top == -INFINITY ? 0.f : top;  // nothing seen yet: adds 0, or a NaN query's NaN
            l_far *= ptx::ex2(z_ref - base);
#pragma unroll
            for (int j = 0; j < 8; ++j) l_far += ptx::ex2(z[j] - base);
            z_ref = top;
          }
          if (mine && !high && q8_far(large)) {  // m may leave z behind from here on
            high = true;
            pt_add(l_far, z_ref, l_run, m_before - kPtShift);
            l_run = 0.f;
          }
        };
        float alpha = 1.f, lsum;
        bool need = false;
        uint32_t pw[32];
        if constexpr (kQ8) {
          bool checked = false, look = m_run == -INFINITY, sum = high;  // sum: kFine, still to be taken
          const float m_before = m_run;
          if (kFine) now = high;
          for (;;) {
            if constexpr (kFine) {
              if (__builtin_expect(__any_sync(0xffffffffu, sum), 0)) sum_far(sum, m_before);
              sum = false;
              read_scores();  // each time: scores, scales and P together do not fit the registers
            }
            if (__builtin_expect(look, 0)) {
              const float tms = tile_max();
              checked = true;
              if (m_run == -INFINITY) {
                m_run = tms;
              } else if (tms > m_run + kPtRescaleLog2) {
                alpha = ptx::ex2(m_run - tms);
                need = true;
                m_run = tms;
              }
            }
            float psum;  // of P: where it is small, no score is far above the reference
            if constexpr (kFine)
              psum = pt_exp64_fine(sv, c, scales, m_run, pw, lsum);
            else
              psum = pt_exp64_q8(sv, gf, ge, m_run, pw, lsum);
            const bool again = !checked && psum >= 128.f * kPtRescaleSum;
            if constexpr (kFine) {
              const bool far = isnan(lsum) && !now;  // or the query is NaN: so is the row either way
              // the warp's rows together; the others' P comes out as it was
              if (!__any_sync(0xffffffffu, again || far)) break;
              if (far) now = sum = true;
            } else if (!again) {
              break;
            }
            look = look || again;
          }
          if (!kFine && __builtin_expect(now || high, 0)) sum_far(true, m_before);
          if (now || high) lsum = 0.f;
        } else {
          bool checked = false;
          if (m_run == -INFINITY) {
            m_run = pt_max64(sv) * c;
            checked = true;
          }
          for (;;) {
            lsum = pt_exp64(sv, c, m_run, pw);
            if (checked || lsum < kPtRescaleSum) break;
            checked = true;
            const float tms = pt_max64(sv) * c;
            if (!(tms > m_run + kPtRescaleLog2)) break;
            alpha = ptx::ex2(m_run - tms);
            need = true;
            m_run = tms;
          }
        }
        ptx::tmem_st32u(colS + buf * kPtKeys, pw);
        if (__any_sync(0xffffffffu, need) && t > 0) {
          // O_X must hold all of PV_X(t - 1) before it is rescaled
          ok = __all_sync(0xffffffffu,
                          pt_wait_for<kShort>(&bars->pv_done[x][(tx - 1) & 1], ((tx - 1) >> 1) & 1, abort_flag));
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll(kShort ? 1 : D / 32)
          for (int c0 = 0; c0 < D; c0 += 32) {
            float ov[32];
            ptx::tmem_ld32(colO + c0, ov);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) ov[k] *= alpha;
            ptx::tmem_st32(colO + c0, ov);
          }
        }
        l_run = l_run * alpha + lsum;
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->p_full[x][buf]);
      }
      // ---- epilogue: every MMA is complete at o_done
      if (nt > 0) {
        ok = ok && __all_sync(0xffffffffu, pt_wait_for<kShort>(&bars->o_done, pieces & 1, abort_flag));
        have_o = ok && ntm > 0;
        if (ok) ptx::tc_fence_after();
      }
      const bool far = l_far != 0.f;
      if (kQ8 && __builtin_expect(__any_sync(0xffffffffu, far), 0)) {
        // m_run becomes the sum's reference and O's with it, half the exponent at a time, as the whole may leave
        // fp32's range
        float f = 1.f;
        if (far) {
          pt_add(l_far, z_ref, l_run, m_run - kPtShift);
          l_run = l_far;
          z_ref += (float)q8_norm(l_run);
          f = ptx::ex2(0.5f * (m_run - kPtShift - z_ref));
          m_run = z_ref + kPtShift;
        }
#pragma unroll 1
        for (int c0 = 0; have_o && c0 < D; c0 += 8) {
          float ov[8];
          ptx::tmem_ld8(colO + c0, ov);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k) ov[k] = ov[k] * f * f;
          ptx::tmem_st8(colO + c0, ov);
          ptx::tmem_wait_st();
        }
      }
      if (isnan(l_run)) m_run = l_run;  // a NaN query's part: no part without a visible key, which merges leave out
      // read here, not kept through the loop
      const volatile PtPiece& at = s_piece[np % kPtPieces];
      const bool whole = kStream && at.c1 <= at.c0;
      const int R = x * kPtRows + r;
      const size_t slot = kStream ? (size_t)at.slot : cta;
      const float inv = whole && l_run > 0.f ? 1.f / l_run : 0.f;
      const size_t orow = (((size_t)b * a.Hq + hk * a.G + g) * a.N + node) * a.D;
      float4* part = whole ? nullptr : reinterpret_cast<float4*>(a.ws_o) + slot * (D / 4) * 2 * kPtRows + R;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        if (x >= pa.tiles) break;
        float ov[32];
        if (have_o) {
          ptx::tmem_ld32(colO + c0, ov);
          ptx::tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) ov[k] = 0.f;
        }
        if (whole) {
          if (valid && c0 < a.D) {
            uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + orow + c0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[k] = make_uint4(ptx::cvt_bf16x2(ov[8 * k + 0] * inv, ov[8 * k + 1] * inv),
                                  ptx::cvt_bf16x2(ov[8 * k + 2] * inv, ov[8 * k + 3] * inv),
                                  ptx::cvt_bf16x2(ov[8 * k + 4] * inv, ov[8 * k + 5] * inv),
                                  ptx::cvt_bf16x2(ov[8 * k + 6] * inv, ov[8 * k + 7] * inv));
          }
        } else {
          // partial O as [D / 4][256 rows] of four columns: a warp stores 512 bytes in a row
#pragma unroll
          for (int k = 0; k < 8; ++k)
            __stcg(part + (size_t)(c0 / 4 + k) * 2 * kPtRows,
                   make_float4(ov[4 * k], ov[4 * k + 1], ov[4 * k + 2], ov[4 * k + 3]));
        }
      }
      if (!whole)
        __stcg(a.ws_ml + slot * 2 * kPtRows + R, make_float2(have_o ? m_run : -INFINITY, have_o ? l_run : 0.f));
      ptx::tc_fence_before();
      __syncwarp();
      if (kStream && nt > 0 && lane == 0) ptx::mbar_arrive(&bars->o_free[x]);
    }
    __syncwarp();

    if constexpr (kStream) {
      // only the softmax warps take part; the others go on to the next piece
      const volatile PtPiece& at = s_piece[np % kPtPieces];
      const int c0 = at.c0, c1 = at.c1;
      if (kWho != kOthers && c0 < c1 && warp >= 2 && warp < 10) {
        __threadfence();
        softmax_sync();
        if (warp == 2 && lane == 0) {
          s_last = ptx::atom_add_acq_rel_gpu(&a.cnt[c0], 1u) == (unsigned)(c1 - c0);
          if (s_last) a.cnt[c0] = 0u;
          __threadfence();
        }
        softmax_sync();
        if (s_last) {
          const int x = (warp - 2) >> 2, r = (hw_warp & 3) * 32 + lane, R = x * kPtRows + r;
          const int g = r / NT, node = pt_of(i0, x) + r % NT;
          if (r < rows_used && node < n_act) {
            auto place = [&](int cc) -> size_t { return cc == c0 ? at.slot0 : 2 * cc; };
            auto stats = [&](int cc) -> float2 { return __ldcg(&a.ws_ml[place(cc) * 2 * kPtRows + R]); };
            float M = -INFINITY, L = 0.f;
#pragma unroll 4
            for (int cc = c0; cc <= c1; ++cc) M = fmaxf(M, stats(cc).x);
#pragma unroll 4
            for (int cc = c0; cc <= c1; ++cc) {
              const float2 ml = stats(cc);
              if (ml.x != -INFINITY) L = fmaf(ptx::ex2(ml.x - M), ml.y, L);
            }
            const float inv = L > 0.f ? 1.f / L : 0.f;
            const size_t orow = (((size_t)b * a.Hq + hk * a.G + g) * a.N + node) * a.D;
#pragma unroll 1
            for (int col = 0; col < a.D; col += 32) {
              float ov[32];
#pragma unroll
              for (int k = 0; k < 32; ++k) ov[k] = 0.f;
              // two parts' loads in flight together
              for (int cc = c0; cc <= c1; cc += 2) {
                float wt[2];
                float4 v[2][8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const int from = min(cc + u, c1);
                  const float2 ml = stats(from);
                  wt[u] = cc + u > c1 || ml.x == -INFINITY ? 0.f : ptx::ex2(ml.x - M);
                  const float4* src = reinterpret_cast<const float4*>(a.ws_o) +
                                      (place(from) * (D / 4) + col / 4) * 2 * kPtRows + R;
#pragma unroll
                  for (int k = 0; k < 8; ++k) v[u][k] = __ldcg(src + (size_t)k * 2 * kPtRows);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                  for (int k = 0; k < 8; ++k) {
                    ov[4 * k] = fmaf(wt[u], v[u][k].x, ov[4 * k]);
                    ov[4 * k + 1] = fmaf(wt[u], v[u][k].y, ov[4 * k + 1]);
                    ov[4 * k + 2] = fmaf(wt[u], v[u][k].z, ov[4 * k + 2]);
                    ov[4 * k + 3] = fmaf(wt[u], v[u][k].w, ov[4 * k + 3]);
                  }
              }
              uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + orow + col);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                dst[k] = make_uint4(ptx::cvt_bf16x2(ov[8 * k + 0] * inv, ov[8 * k + 1] * inv),
                                    ptx::cvt_bf16x2(ov[8 * k + 2] * inv, ov[8 * k + 3] * inv),
                                    ptx::cvt_bf16x2(ov[8 * k + 4] * inv, ov[8 * k + 5] * inv),
                                    ptx::cvt_bf16x2(ov[8 * k + 6] * inv, ov[8 * k + 7] * inv));
            }
          }
        }
      }
    } else {
      // the parts form one cluster, and each CTA merges its share of the rows.  They meet in L2, not in
      // distributed shared memory: 64 KB a CTA through a cluster took 2.8 us, stored or read
      ptx::cluster_sync();
      const int S = pa.splits;
      const int share = (pa.tiles * kPtRows + S - 1) / S;
      const int r0 = split * share, rows = min(pa.tiles * kPtRows, r0 + share) - r0;
      const size_t first = cta - split;
      for (int item = threadIdx.x; item < rows * (a.D / 4); item += C::kThreads) {
        const int ch = item / rows, R = r0 + item - ch * rows;
        const int x = R >= kPtRows ? 1 : 0, r = R - x * kPtRows;
        const int g = r / NT, node = pt_of(i0, x) + r % NT;
        if (r >= rows_used || node >= n_act) continue;
        float2 mlv[kPtMaxSplits];
        float4 xv[kPtMaxSplits];
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int s2 = 0; s2 < kPtMaxSplits; ++s2)
          if (s2 < S) {
            mlv[s2] = __ldcg(a.ws_ml + (first + s2) * 2 * kPtRows + R);
            xv[s2] = __ldcg(reinterpret_cast<const float4*>(a.ws_o) + ((first + s2) * (D / 4) + ch) * 2 * kPtRows + R);
          }
#pragma unroll
        for (int s2 = 0; s2 < kPtMaxSplits; ++s2)
          if (s2 < S) M = fmaxf(M, mlv[s2].x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s2 = 0; s2 < kPtMaxSplits; ++s2)
          if (s2 < S && mlv[s2].x != -INFINITY) {
            const float w = ptx::ex2(mlv[s2].x - M);
            L = fmaf(mlv[s2].y, w, L);
            acc.x = fmaf(w, xv[s2].x, acc.x);
            acc.y = fmaf(w, xv[s2].y, acc.y);
            acc.z = fmaf(w, xv[s2].z, acc.z);
            acc.w = fmaf(w, xv[s2].w, acc.w);
          }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const size_t o = (((size_t)b * a.Hq + hk * a.G + g) * a.N + node) * a.D + ch * 4;
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + o) =
            make_uint2(ptx::cvt_bf16x2(acc.x * inv, acc.y * inv), ptx::cvt_bf16x2(acc.z * inv, acc.w * inv));
      }
    }
    if constexpr (kStream) {
      __syncwarp();
      if (warp != 0 && lane == 0) ptx::mbar_arrive(&bars->piece_empty[np % kPtPieces]);
    }
    kt += nt;
    rounds += (nt + 7) / 8;
    done_x[0] += ntx[0];
    done_x[1] += ntx[1];
    pieces += nt > 0;
    if (!kStream) break;
  }
  if (kStream && warp == 0 && lane == 0) drain();
  };
  if constexpr (kQ8) {
    if (warp >= 2 && warp < 10) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
      run_pieces(std::integral_constant<int, kSoftmax>());
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
      run_pieces(std::integral_constant<int, kOthers>());
    }
  } else {
    run_pieces(std::integral_constant<int, kAll>());
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && bars->abort) set_dev_status(a.dev_status, TV_DEV_TIMEOUT);
}

// ---- host side

template <int D, int kCap, bool kStream, int kQ>
static cudaError_t launch_pt(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a,
                             const PtPlan& p, cudaStream_t stream) {
  using C = PtCfg<D, kQ>;
  constexpr int smem = C::kSmemAlloc;
  const auto fn = paged_tc_kernel<D, kCap, kStream, kQ>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const PtArgs pa{p.NT, p.tiles, p.MP, p.splits, a.D == 128};
  if (kStream)
    return launch_pdl(fn, dim3((unsigned)p.grid), dim3(C::kThreads), smem, stream,
                      nullptr, 0, mq, mk, mv, a, pa);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  return launch_pdl(fn, dim3((unsigned)(p.MP * p.splits), (unsigned)a.Hkv, (unsigned)a.B),
                    dim3(C::kThreads), smem, stream, attr, 1, mq, mk, mv, a, pa);
}

template <int D, int kCap, int kQ>
static cudaError_t launch_pt_c(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a,
                               const PtPlan& p, cudaStream_t stream) {
  return p.splits ? launch_pt<D, kCap, false, kQ>(mq, mk, mv, a, p, stream)
                  : launch_pt<D, kCap, true, kQ>(mq, mk, mv, a, p, stream);
}
template <int D, int kQ>
static cudaError_t launch_pt_d(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttn& a,
                               const PtPlan& p, cudaStream_t stream) {
  switch (cap_mode(a.cap)) {
    case kLargeCap:
      return launch_pt_c<D, kLargeCap, kQ>(mq, mk, mv, a, p, stream);
    case kTanhCap:
      return launch_pt_c<D, kTanhCap, kQ>(mq, mk, mv, a, p, stream);
    default:
      return launch_pt_c<D, kNoCap, kQ>(mq, mk, mv, a, p, stream);
  }
}

template <int kQ>
static cudaError_t launch_pt_all(PagedAttn a, char* ws, cudaStream_t stream) {
  const PtPlan p = paged_tc_plan(a.B, a.Hq, a.Hkv, a.D, a.N, a.sms);
  a.cnt = reinterpret_cast<unsigned*>(ws);
  a.ws_ml = reinterpret_cast<float2*>(ws + kPagedCntBytes);
  a.ws_o = reinterpret_cast<float*>(ws + kPagedCntBytes + p.slots * 2 * kPtRows * 8);
  CUtensorMap mq, mk, mv;
  const bool made = kQ != kPtBf16 ? paged_q8_tmap(&mk, a.k, a, kQ8Rows128, a.D == 96 ? 8 : 64) && paged_q8_tmap(&mv, a.v, a, kQ8Plain)
                        : paged_q_tmap(&mq, a, p.NT) && paged_kv_tmap(&mk, a.k, a) && paged_kv_tmap(&mv, a.v, a);
  if (!made) return cudaErrorInvalidValue;
  if (kQ != kPtBf16) mq = mk;  // Q comes without one
  return a.D <= 64 ? launch_pt_d<64, kQ>(mq, mk, mv, a, p, stream) : launch_pt_d<128, kQ>(mq, mk, mv, a, p, stream);
}

}  // namespace tv
