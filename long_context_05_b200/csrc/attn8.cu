// Sparse and dense MQA/MLA attention over an 8-bit latent cache, on tcgen05.
//
// The cache holds one e4m3 row k8 of d_k bytes and one FP32 scale s per token,
// shared by all heads; the value is the row's first d_v columns.  With
// a = tau log2(e):
//   x_k = a s_k (q . k8_k) + log2 s_k,        R a running reference,
//   P_k = 2^(x_k - R) = 2^(logit_k - R) s_k,  l = sum_k P_k / s_k,
//   out = sum_k P_k k8_k[:d_v] / l,           lse = (R + log2 l) ln 2
// (s_k outside a in units of a power of two near the first key's).
// The token's scale is folded into the exponent, so the cached bytes go to
// the tensor cores as they are, in both products: no dequantised copy of a
// key exists anywhere, a key costs 576 bytes of shared memory instead of
// 1152, and the gather moves half the bytes of the BF16 cache.
//
// kind::f8f6f4 multiplies 8-bit floats at twice the BF16 rate, so the other
// operand is split in two 8-bit terms and every product runs twice, at the
// cost of one BF16 product:
//   * q = 2^e (q_hi + q_lo), both e4m3, 2^e per head row with max|q| <= 448 *
//     2^e.  A BF16 number has 8 significant bits and e4m3 four, so the two
//     terms give q exactly down to 2^-10 of the row's largest, and within
//     2^-17.8 of it below (half of e4m3's subnormal step over 224);
//   * P = P_hi (e4m3) + P_lo (e5m2): off by 2^-8 of P at worst, as one BF16
//     number, and 2^-9.6 in the mean square, down to P = 2^-6, and by 2^-14
//     or less below.  (With P_lo in e4m3, as precise again above, what lies
//     below 2^-10 was lost: a tail of 8191 keys ten nats under one key a
//     quarter of the output.)
// So that 2^-14 stays small beside what a row holds, however long it is, R
// keeps the largest P of a row between 2^kHead and 2^kTop: 2048 keys lose at
// most 2048 * 2^-14 / 2^kHead = 2^-9 of the largest one.  Where a part has
// more keys, R also comes down when the largest P of a chunk falls below
// 2^(kHead - kDrop): a chunk then loses at most 128 * 2^-14 / 2^(kHead -
// kDrop) = 2^-9 of its own largest.  The accumulator, FP32, has the range for
// that; kDepth bounds how far R lies under the highest it ever was.
// Logits, P before its rounding, l and the output accumulate in FP32.
//
// Work split.  A CTA takes 64 head rows and all value columns: heads of one
// query, or in a dense call, where the queries of a sequence share their keys,
// rows of the sequence's T x H (several queries where there are few heads,
// with the keys past a row's own position masked in its logits; 1538 dense
// queries over up to 1537 keys took 225 us at 8 heads and 480 at 72 with a
// query to a CTA, 50 and 292 so, and the same at 64 and 128).  They are the M = 64 of tcgen05.mma.ws: that form
// spreads a 64 x N result over all 128 TMEM lanes (lanes 0-63 the first N/2
// columns, 64-127 the rest), so the 64 x 512 FP32 accumulator takes half of
// TMEM.  With M = 128 it would fill TMEM, and the way out, a CTA per half of
// the value columns, computes every logit twice.  Measured, back to back:
// N = 128 45-49 cycles, N = 256 77-82 (M = 128: 64 and 129), so a query's
// 128 keys cost 2 x 3000 cycles of MMAs in place of 2 x 4400 (M = 128 with the
// N = 64 that fits beside the accumulator).  Few head rows also split their
// keys, and a combine kernel merges the parts.
//
// Per CTA: TMEM holds O (256 columns) | two S buffers of 64 | q_hi and q_lo of
// the first 256 key columns, in both lane halves.  Shared memory holds the
// rest of q (40 KB), two regions of 128 keys (144 KB) and two P buffers.
// Chunks a, b of 128 keys alternate between the regions, and the tensor core
// gets q K^T(a), q K^T(b), P V(a), P V(b): the softmax of a runs under
// q K^T(b), that of b under P V(a), and the next a is gathered under P V(b),
// the next b under q K^T.
// Warp roles (576 threads): warp 0 issues the MMAs; warp 1 forms the per-key
// constants; warps 2-9 are the softmax, warps 10-17 gather 16 keys each with
// 16-byte cp.async that arrive on the region's barrier by themselves.  Four
// softmax threads share a head row (32 keys each) and exchange their maxima
// through shared memory.  When R moves, the accumulator is rescaled once.
//
// Measured (576 / 512).  2048 queries of 128 heads over 2048 selected keys
// each: 1290 to 1320 us kept up for seconds, at the board's power limit (885 to
// 905 TFLOP/s of the 1168 GFLOP counted once; the two terms count double on
// the tensor cores), 1120 us back to back before it sets in.  A CTA takes
// 72800 cycles, and the next 1400 more to start.  To its first logits 10300,
// 7900 of them until q lies in place (150 KB of q and keys at 27 bytes a clock
// from L2 with every SM asking; a third fewer instructions in q's split
// changed nothing); then 7400 for two chunks, with keys of one norm 6475 of
// MMAs and 925 of waiting for the second chunk's softmax, which is longer than
// the P V it runs under; from the last P V to the last store 2500 (the stores'
// way out), and 1100 to its end.  Sixteen softmax warps were slower (1575 us:
// the MMA warp lost issue slots), and so were CTAs that stay and place the
// next tile's q under the end of the last (1150 us for 1160 then, but dense
// calls 515 for 444: the hardware's own order of unequal CTAs is better, and
// the split slows the output down).  A decode step of 8 x 128 heads over 2048
// keys: 16.8 us with the combine.  A selection leaves a CTA the heads of one
// query: with 8 heads an eighth of its rows is used, with 72 nine in sixteen.
#include <cuda_fp8.h>
#include <math.h>

#include "internal.h"
#include "sm100.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kN = 128;                // keys per chunk
constexpr int kM = 64;                 // heads per CTA
constexpr int kMmaWarp = 0, kParamWarp = 1, kFirstSoftmax = 2, kFirstGather = 10, kGatherWarps = 8;
constexpr int kThreads = 32 * (kFirstGather + kGatherWarps);
constexpr uint32_t kTmemCols = 512;
constexpr float kHead = 6.f;           // log2 of the largest P of a row when R is set (P is then exact)
constexpr float kTop = 8.75f;          // ... and at most (2^8.75 < 448)
// (With kHead 4, 5, 6 and 8, on keys of spread norms, R moves in 9.1, 9.7, 10.4
// and 12.3 of 15 chunks of a warp: 1114, 1119 and 1123 us with 4, 5 and 6 on
// 2048 queries of 128 heads over 2048 keys.)
constexpr float kDrop = 4.f;           // how far a chunk's maximum may fall short of kHead
constexpr int kLongPart = 2048;        // in parts of more keys than this
constexpr float kDepth = 24.f;         // how far R may come down from the highest it was

template <int DK, int DV>
struct Cfg {
  static constexpr int KSTEPS = (DK + 31) / 32;        // 32-byte MMA K steps
  static constexpr int NF = DK >= 128 ? DK / 128 : 1;  // 128-byte atoms of a row
  static constexpr int TAIL = DK > NF * 128 ? 1 : 0;   // one 64-byte atom more
  static constexpr int NV = DV < 256 ? DV : 256;       // value columns of one MMA
  static constexpr int NMMV = DV / NV;
  static constexpr int OCOLS = DV / 2;                 // TMEM columns of the accumulator
  static constexpr uint32_t OCOL = 0;
  static constexpr uint32_t SCOL = 256;
  static constexpr uint32_t QCOL = SCOL + 2 * (kN / 2);
  static constexpr int QT = DK > 256 ? 256 : 0;        // leading key columns whose q lies in TMEM
  static constexpr int QSF = NF - QT / 128;            // q atoms in shared memory
  static constexpr int QPIECE = QSF * kM * 128 + TAIL * kM * 64;
  static constexpr int ATOM = 2 * kN * 128;            // bytes of one atom of both regions
  static constexpr int KV_BYTES = NF * ATOM + TAIL * 2 * kN * 64;
  static constexpr int PTERM = kM * kN;                // bytes of one term of a P buffer
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = (2 * QPIECE + 1023) / 1024 * 1024;
  static constexpr int OFF_P = OFF_KV + KV_BYTES;      // [2][hi, lo][64 rows x 128 bytes]
  static constexpr int OFF_PAR = OFF_P + 4 * PTERM;    // [2][3][128]: a s, log2 s, 1 / s of the keys
  static constexpr int OFF_MX = OFF_PAR + 2 * kN * 12; // [2][4][64] partial maxima
  static constexpr int OFF_E = OFF_MX + 2 * 4 * kM * 4;  // [64] 2^e of the head rows
  static constexpr int OFF_BAR = OFF_E + kM * 4;
  static constexpr int NBARS = 1 + 2 + 4 + 2 + 2 + 2 + 2 + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBARS * 8;   // TMEM's base, abort flag, scale unit
  static constexpr int BYTES = OFF_MISC + 16;
  static_assert(BYTES <= 232448, "shared memory per CTA");
  static_assert(OFF_KV % 1024 == 0 && OFF_P % 1024 == 0 && OFF_BAR % 8 == 0, "alignment");
  static_assert(OCOLS <= 256 && QCOL + 2 * (QT / 4) <= kTmemCols, "TMEM");
  // q's bytes on their way to TMEM pass through the P buffers
  static_assert(2 * QT * kM <= 4 * PTERM, "staging");
};

// n / d for 0 <= n < 2^31 as a product with 2^32 (2^s / d - 1) rounded up, s
// the first with 2^s >= d (Granlund and Montgomery): five divisions by every
// warp of a CTA took 1200 cycles of its start.
struct Divisor {
  uint32_t mul, shift;
  static Divisor of(int d) {
    Divisor r{0, 0};
    while ((1ull << r.shift) < (unsigned)d) ++r.shift;
    r.mul = (uint32_t)(((1ull << 32) * ((1ull << r.shift) - (unsigned)d)) / (unsigned)d + 1);
    return r;
  }
  __device__ __forceinline__ int operator()(int n) const {
    return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
  }
};

struct Params {
  KvMap map;
  const uint16_t* q;
  const uint8_t* kv8;
  const float* kv_scale;
  const int32_t* idx;    // null: every row dense
  int dense_rows;        // rows with t < dense_rows take keys 0..pos(t), idx unread
  uint16_t* out;
  float* lse;
  // nsplit > 1: the parts' outputs, normalised by their own l, as FP16 times
  // one FP32 factor per 32 columns (16 at d_v 64): a group's largest is 2^14
  // or more, so its values keep FP16's 11 bits down to 2^-28 of it, whatever
  // the cache's scales
  __half* part_o;        // [rows, nsplit, H, d_v]
  float* part_f;         // [rows, nsplit, H, d_v / 32 (16)]
  float* part_lse;       // [rows, nsplit, H], log2 units
  int T, H, k;
  // A unit is one query, with its H head rows, or in a dense call one
  // sequence, with all its T H; a CTA takes 64 head rows of one.
  int units, HR, nsplit, hsplit;
  Divisor by_T, by_H, by_nsplit, by_hsplit;
  int ahead;             // CTAs of a wave: the next on this SM is about so many on
  float scale_log2;      // tau log2(e)
  long long wait_ns;
  DevErr* err;
};

__device__ __forceinline__ int pow2_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, -126), 120);
}
template <__nv_fp8_interpretation_t TO>
__device__ __forceinline__ uint32_t fp8x2_of_half2(__half2 h) {
  return (uint32_t)__nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<__half2_raw*>(&h), __NV_SATFINITE, TO);
}
__device__ __forceinline__ __half2 half2_of_e4m3x2(uint32_t v) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)v, __NV_E4M3));
}
// two terms of a pair of numbers (|a|, |b| <= 448), e4m3 and LO: low 16 bits of hi, lo
template <__nv_fp8_interpretation_t LO>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  hi = fp8x2_of_half2<__NV_E4M3>(h);
  lo = fp8x2_of_half2<LO>(__hsub2(h, half2_of_e4m3x2(hi)));
}

// D[tmem] (+)= A B^T, 8-bit floats, the M = 64 form that uses all lanes; A in shared
// memory or in TMEM (in lanes 0-63 and again in 64-127).  The two terms of A
// meet the same B one after the other: the first MMA leaves B in the
// collector and the second takes it from there, which halves the reads of
// shared memory (1200 -> 1170 us on 2048 queries of 128 heads).
template <int TERM>
__device__ __forceinline__ void mma_ws(uint32_t d_tmem, uint64_t a, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (TERM == 0) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.ws.cta_group::1.kind::f8f6f4.collector::b0::fill [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.ws.cta_group::1.kind::f8f6f4.collector::b0::lastuse [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
template <int TERM>
__device__ __forceinline__ void mma_ws_ts(uint32_t d_tmem, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  if constexpr (TERM == 0) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.ws.cta_group::1.kind::f8f6f4.collector::b0::fill [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.ws.cta_group::1.kind::f8f6f4.collector::b0::lastuse [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void prefetch_l2(const void* a) { asm volatile("prefetch.global.L2 [%0];" ::"l"(a)); }

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// largest magnitude of eight BF16 numbers, as its bits
__device__ __forceinline__ uint32_t max_abs8(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  return m;
}

// W columns of TMEM times alpha (32 lanes of one warp), 64 in flight
template <int W>
__device__ __forceinline__ void tmem_scale(uint32_t addr, float alpha) {
  if constexpr (W >= 64) {
#pragma unroll 1
    for (int x = 0; x < W; x += 64) {
      uint32_t o0[32], o1[32];
      tmem_ld32(addr + x, o0);
      tmem_ld32(addr + x + 32, o1);
      tmem_wait_ld_dep(o0);
      tmem_wait_ld_dep(o1);
#pragma unroll
      for (int i = 0; i < 32; ++i) o0[i] = __float_as_uint(__uint_as_float(o0[i]) * alpha);
      tmem_st32(addr + x, o0);
#pragma unroll
      for (int i = 0; i < 32; ++i) o1[i] = __float_as_uint(__uint_as_float(o1[i]) * alpha);
      tmem_st32(addr + x + 32, o1);
    }
  } else {
    static_assert(W == 16, "columns");
    uint32_t o[16];
    tmem_ld16(addr, o);
    tmem_wait_ld_dep(o);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
    tmem_st16(addr, o);
  }
  tmem_wait_st();
}

// R head rows of q (rows r0 .. r0 + R - 1 of the CTA's 64) in two e4m3 terms,
// by one warp.  A step is 32 vectors of eight columns: the full steps of each
// row, then what is left of the rows' columns, 32 / RV rows to a step, so that
// a lane's place in shared memory is known once for all rows but for the
// swizzle.  A row's exponent comes from its maximum over the warp.
template <int DK, int R>
struct QRows {
  static constexpr int FULL = DK / 256;                  // full steps of a row
  static constexpr int DIV = FULL > 0 ? FULL : 1;
  static constexpr int RV = (DK - FULL * 256) / 8 <= 8 ? 8 : 16;   // lanes of a row in the last steps
  static constexpr int TAILS = (R * RV + 31) / 32;       // last steps
  static constexpr int STEPS = R * FULL + TAILS;
  uint4 v[STEPS];
  __device__ __forceinline__ void load(const uint16_t* q, int heads, int r0, int lane) {
    const uint16_t* q0 = q + (size_t)r0 * DK;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const bool full = s < R * FULL;
      const int row = full ? s / DIV : (s - R * FULL) * (32 / RV) + lane / RV;
      const int col = full ? s % DIV * 256 + lane * 8 : FULL * 256 + (lane % RV) * 8;
      v[s] = make_uint4(0u, 0u, 0u, 0u);
      if (row < R && r0 + row < heads && col < DK) v[s] = __ldg(reinterpret_cast<const uint4*>(q0 + row * DK + col));
    }
  }
};
template <int DK, int DV, int R>
__device__ __forceinline__ void split_q_rows(const QRows<DK, R>& q4, int r0, int lane, uint8_t* sQ, uint8_t* sP,
                                             float* sE) {
  using C = Cfg<DK, DV>;
  using Q = QRows<DK, R>;
  uint32_t m[R] = {};
#pragma unroll
  for (int s = 0; s < Q::STEPS; ++s) {
    const uint32_t x = max_abs8(q4.v[s]);
    if (s < R * Q::FULL) {
      m[s / Q::DIV] = max(m[s / Q::DIV], x);
    } else {
#pragma unroll
      for (int i = 0; i < 32 / Q::RV; ++i) {
        const int row = (s - R * Q::FULL) * (32 / Q::RV) + i;
        if (row < R) m[row] = max(m[row], lane / Q::RV == i ? x : 0u);
      }
    }
  }
  float inv[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const uint32_t most = __reduce_max_sync(0xffffffffu, m[i]);
    const int e = pow2_exponent(__uint_as_float(most << 16));
    inv[i] = __uint_as_float((uint32_t)(127 - e) << 23);
    // a row with an infinity or a NaN has NaN logits (e4m3 has no infinity)
    if (lane == i) sE[r0 + i] = most >= 0x7f80u ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)(127 + e) << 23);
  }
  // both terms of eight columns: 8 bytes at d and at d + to_lo
  auto put = [&](const uint4& v, float f, uint8_t* d, int to_lo) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int y = 0; y < 4; ++y)
      split2<__NV_E4M3>(__uint_as_float(x[y] << 16) * f, __uint_as_float(x[y] & 0xffff0000u) * f, hi[y], lo[y]);
    *reinterpret_cast<uint2*>(d) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
    *reinterpret_cast<uint2*>(d + to_lo) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
  };
#pragma unroll
  for (int s = 0; s < Q::STEPS; ++s) {
    if (s < R * Q::FULL) {
      const int i = s / Q::DIV, u = s % Q::DIV, rr = r0 + i;
      const int c16 = (lane & 15) >> 1, in_atom = (lane >> 4) * (kM * 128);
      const int at = rr * 128 + ((c16 ^ (rr & 7)) << 4) + (lane & 1) * 8 + in_atom;
      // q's TMEM columns are staged in the P buffers: [term][atom][64 rows x 128 bytes]
      if (u * 256 < C::QT) put(q4.v[s], inv[i], sP + (u * 2) * (kM * 128) + at, (C::QT / 128) * (kM * 128));
      else put(q4.v[s], inv[i], sQ + (u * 2 - C::QT / 128) * (kM * 128) + at, C::QPIECE);
    } else {
      const int i = (s - R * Q::FULL) * (32 / Q::RV) + lane / Q::RV, rr = r0 + i, l = lane % Q::RV;
      if (i >= R || Q::FULL * 256 + l * 8 >= DK) continue;
      float f = inv[0];
#pragma unroll
      for (int y = 1; y < R; ++y) f = i == y ? inv[y] : f;
      uint8_t* d = C::TAIL != 0 ? sQ + C::QSF * (kM * 128) + rr * 64 + (((l >> 1) ^ ((rr >> 1) & 3)) << 4)
                                : sQ + rr * 128 + (((l >> 1) ^ (rr & 7)) << 4);
      put(q4.v[s], f, d + (l & 1) * 8, C::QPIECE);
    }
  }
}

template <int DK, int DV, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) attn8_kernel(Params p) {
  using C = Cfg<DK, DV>;
  extern __shared__ uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    // self-check: the swizzled layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) report_error(p.err, DSA_ERR_DEVICE_BOUNDS, ERR_SITE_ATTN8 | (0xAu << 8));
    return;
  }
  // what follows on the stream may be scheduled now (the combine, or another
  // call's kernel: both wait for this grid before they touch memory), and this
  // kernel waits for what was before it
  pdl_launch_dependents();
  pdl_wait();
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sKV = smem + C::OFF_KV;
  uint8_t* sP = smem + C::OFF_P;
  float* sPar = reinterpret_cast<float*>(smem + C::OFF_PAR);
  float* sMx = reinterpret_cast<float*>(smem + C::OFF_MX);
  float* sE = reinterpret_cast<float*>(smem + C::OFF_E);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_ready = bars;                    // q in shared memory and TMEM (8 softmax warps)
  uint64_t* kv_full = q_ready + 1;             // [region] rows landed (8 gather warps, every lane)
  uint64_t* kv_empty = kv_full + 2;            // [region][half] P V of the half's keys complete (commit)
  uint64_t* par_full = kv_empty + 4;           // [2] per-key constants written (32 lanes)
  uint64_t* par_empty = par_full + 2;          // [2] and read (8 warps)
  uint64_t* s_full = par_empty + 2;            // [2] q K^T complete (commit)
  uint64_t* p_full = s_full + 2;               // [2] P written (8 warps)
  uint64_t* mma_done = p_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  float* sUnit = reinterpret_cast<float*>(smem + C::OFF_MISC + 8);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const bool packed = p.idx == nullptr;        // units are sequences
  // head rows [64 hs, 64 hs + 64) of the unit; in a dense call the last
  // queries, of the most keys, first
  const int rest = p.by_hsplit(blockIdx.x), br = (int)blockIdx.x - rest * p.hsplit;
  const int hs = packed ? p.hsplit - 1 - br : br;
  const int unit = p.by_nsplit(rest);          // b * T + t, or b
  const int split = rest - unit * p.nsplit;
  const int b = packed ? unit : p.by_T(unit);
  const int nrows = min(kM, p.HR - hs * kM);
  const int t = packed ? p.by_H(hs * kM + nrows - 1) : unit - b * p.T;   // the last query of the rows
  const int Lb = p.map.len(b, threadIdx.x == 0 ? p.err : nullptr, ERR_SITE_ATTN8);
  const bool dense = packed || t < p.dense_rows;
  const int nslots = dense ? Lb - p.T + t + 1 : p.k;      // slots of these rows
  // an equal share of the row's chunks for every split
  const int kc = p.by_nsplit((nslots + kN - 1) / kN + p.nsplit - 1) * kN;
  const int slot0 = min(split * kc, nslots), slot1 = min(slot0 + kc, nslots);
  const int nchunks = (slot1 - slot0 + kN - 1) / kN;

  const int32_t* irow = dense ? nullptr : p.idx + (size_t)unit * p.k;
  // index of slot s of this split; -1 past the end and for an empty slot
  auto load_idx = [&](int s) -> int { return s < slot1 ? (dense ? s : irow[s]) : -1; };
  // q's rows are on their way while the barriers are set up: six to a softmax
  // warp, from the first, and two to a gather warp, behind its first chunk
  // (four to each: the softmax warps waited 2500 cycles for the others)
  const int kl = 16 * (warp - kFirstGather) + (lane & 15);
  int i_cur = -1, i_next = -1;
  if (warp >= kFirstGather) {
    i_cur = load_idx(slot0 + kl);
    i_next = load_idx(slot0 + kN + kl);
  }
  const uint16_t* q0 = p.q + ((size_t)unit * p.HR + hs * kM) * DK;
  QRows<DK, 4> q4;
  QRows<DK, 2> q2;                             // rows 32..47, 48..63
  if (warp >= kFirstSoftmax) {
    if (warp < kFirstGather) q4.load(q0, nrows, 4 * (warp - kFirstSoftmax), lane);
    q2.load(q0, nrows, 32 + 2 * (warp - kFirstSoftmax), lane);
  }

  if (warp == kParamWarp) {
    // a lane's barrier (they lie side by side in this order) and its arrivals
    const int i = lane;
    const uint32_t arrivals = i == 0 ? 8                       // q_ready
                              : i < 3 ? 32 * kGatherWarps      // kv_full
                              : i < 7 ? 1                      // kv_empty
                              : i < 9 ? 32                     // par_full
                              : i < 11 ? 8                     // par_empty
                              : i < 13 ? 1                     // s_full
                              : i < 15 ? 8                     // p_full
                                       : 1;                    // mma_done
    if (i < C::NBARS) mbar_init(bars + i, arrivals);
    if (i == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if constexpr (DK % 128 != 0 && C::TAIL == 0) {
    // columns DK.. of the atoms of q (rows 0..127: both terms) and of the keys
    for (int i = threadIdx.x; i < 2 * (kM + kN) * 8; i += kThreads) {
      const int rr = i / 8;
      uint8_t* d = rr < 2 * kM ? sQ + rr * 128 : sKV + (rr - 2 * kM) * 128;
      if (i % 8 >= DK / 16) *reinterpret_cast<uint4*>(d + (((i % 8) ^ (rr & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  __syncthreads();
  // TMEM is not needed before q is split: its allocation, 2000 cycles, runs
  // beside the first gather, and barrier 1 tells the softmax warps
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
    tc_fence_before();
    asm volatile("bar.arrive 1, 544;" ::: "memory");
  }
  auto tmem_base = [&]() -> uint32_t {
    tc_fence_after();
    return __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(tmem_slot), 0);
  };

  const AbortSources ab{abort_flag, &p.err->code};
  const AbortSources no_abort{nullptr, nullptr};
  auto fail = [&](unsigned where) {
    report_error(p.err, DSA_ERR_TIMEOUT, ERR_SITE_ATTN8 | (where << 8));
    *abort_flag = 1;
  };
  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
    const bool r = mbar_wait(bar, parity, p.wait_ns, ab);
    return __all_sync(0xffffffffu, r);
  };
  // cache row (relative to the sequence's first in a contiguous cache); -1
  // for no key and for an index outside [0, L_b)
  auto row_of = [&](int v) -> int {
    if (v < 0 || v >= Lb) return -1;
    return PAGED ? (int)p.map.row<true>(b, v) : v;
  };
  const long long base_row = PAGED ? 0 : (long long)b * p.map.S;

  if (warp >= kFirstGather) {
    // ------------------------------------------------------------ gather
    // warp g copies keys [16 g, 16 g + 16) of every chunk
    const int g = warp - kFirstGather;
    const uint8_t* base = p.kv8 + base_row * DK;
    int r_cur = row_of(i_cur);
    // this warp's rows of q, behind the first chunk
    auto help_q = [&]() {
      split_q_rows<DK, DV>(q2, 48 + 2 * g, lane, sQ, sP, sE);
      fence_proxy_async_smem();
      asm volatile("bar.arrive 1, 544;" ::: "memory");
    };
    for (int j = 0; j < nchunks; ++j) {
      const int rg = j & 1;
      if (j >= 2 && !wwait(&kv_empty[2 * rg + g / 4], (uint32_t)(j / 2 - 1) & 1)) { fail(1); break; }
      const int r_next = row_of(i_next);
      i_next = load_idx(slot0 + (j + 2) * kN + kl);
      uint8_t* dst0 = sKV + (rg * kN + 16 * g) * 128;
      const int c = lane & 7, k8 = lane >> 3;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int kr = 4 * m + k8;                       // key within the warp's 16
        const int r = __shfl_sync(0xffffffffu, r_cur, kr);
        const uint8_t* src = base + (size_t)(r < 0 ? 0 : r) * DK + c * 16;
        uint8_t* dst = dst0 + kr * 128 + ((c ^ (kr & 7)) << 4);
#pragma unroll
        for (int a = 0; a < C::NF; ++a)
          if (a * 128 + c * 16 < DK) cp_async16_zfill(dst + a * C::ATOM, src + a * 128, r < 0 ? 0u : 16u);
      }
      if constexpr (C::TAIL != 0) {
        const int c4 = lane & 3, k4 = lane >> 2;
        uint8_t* tail0 = sKV + C::NF * C::ATOM + (rg * kN + 16 * g) * 64;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int kr = 8 * m + k4;
          const int r = __shfl_sync(0xffffffffu, r_cur, kr);
          cp_async16_zfill(tail0 + kr * 64 + ((c4 ^ ((kr >> 1) & 3)) << 4),
                           base + (size_t)(r < 0 ? 0 : r) * DK + C::NF * 128 + c4 * 16, r < 0 ? 0u : 16u);
        }
      }
      cp_async_arrive(&kv_full[rg]);
      r_cur = r_next;
      if (j == 0) help_q();
    }
    if (nchunks == 0) help_q();
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == kParamWarp) {
    // ------------------------------------------------------------ per-key constants
    // lane l holds keys l, l + 32, l + 64, l + 96 of a chunk
    auto scale_of = [&](int r) -> float { return r < 0 ? 0.f : __ldg(p.kv_scale + base_row + r); };
    auto checked_row = [&](int v) -> int {
      if (v >= Lb) {
        report_error(p.err, DSA_ERR_DEVICE_BOUNDS, ERR_SITE_ATTN8);
        return -1;
      }
      const int r = row_of(v);
      if (PAGED && v >= 0 && r < 0) report_error(p.err, DSA_ERR_DEVICE_BOUNDS, ERR_SITE_ATTN8 | (1u << 8));
      return r;
    };
    // the rows of q, and of indices, that the next CTA on this SM begins with,
    // on their way to L2
    const int x = (int)blockIdx.x + p.ahead;
    if (x < (int)gridDim.x) {
      const int rest2 = p.by_hsplit(x), br2 = x - rest2 * p.hsplit, unit2 = p.by_nsplit(rest2);
      const int hs2 = packed ? p.hsplit - 1 - br2 : br2;
      const char* q2 = reinterpret_cast<const char*>(p.q + ((size_t)unit2 * p.HR + hs2 * kM) * DK);
      for (int i = lane * 128; i < min(kM, p.HR - hs2 * kM) * DK * 2; i += 32 * 128) prefetch_l2(q2 + i);
      if (!packed)
        for (int i = lane * 32; i < p.k; i += 32 * 32) prefetch_l2(p.idx + (size_t)unit2 * p.k + i);
    }
    int ip[4];
    float s_cur[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) ip[u] = load_idx(slot0 + lane + 32 * u);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      s_cur[u] = scale_of(checked_row(ip[u]));
      ip[u] = load_idx(slot0 + kN + lane + 32 * u);
    }
    float unit = 1.f, unit_log2 = 0.f;
    for (int j = 0; j < nchunks; ++j) {
      float s_next[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        s_next[u] = scale_of(checked_row(ip[u]));
        ip[u] = load_idx(slot0 + (j + 2) * kN + lane + 32 * u);
      }
      if (j == 0) {
        // Scales count in units of the first key's (of the first 32 slots, or
        // the chunk's largest; rows of a CTA share their first keys), so that
        // how far l is from 1 does not depend on the scales but on their spread.
        const uint32_t some = __ballot_sync(0xffffffffu, s_cur[0] > 0.f);
        const uint32_t s0 =
            some != 0u ? __shfl_sync(0xffffffffu, __float_as_uint(s_cur[0]), __ffs((int)some) - 1)
                       : __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(s_cur[1], fmaxf(s_cur[2], s_cur[3]))));
        if (s0 >= 0x00800000u) unit = __uint_as_float(s0 & 0x7f800000u);
        unit_log2 = (float)((int)(__float_as_uint(unit) >> 23) - 127);
        if (lane == 0) *sUnit = unit;
      }
      const int pb = j & 1;
      if (j >= 2 && !wwait(&par_empty[pb], (uint32_t)(j / 2 - 1) & 1)) { fail(3); break; }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float s = s_cur[u];
        const bool on = s > 0.f;
        float* par = sPar + pb * 3 * kN + lane + 32 * u;
        par[0] = p.scale_log2 * s;
        par[kN] = on ? log2f(s) - unit_log2 : -INFINITY;
        par[2 * kN] = on ? fminf(unit / s, 3.0e38f) : 0.f;   // (finite: it may meet a P of zero)
        s_cur[u] = s_next[u];
      }
      mbar_arrive(&par_full[pb]);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    // the whole warp runs this code and one elected lane issues, so that the
    // descriptors stay in uniform registers: a lane alone on its branch took
    // 80 cycles an MMA, more than the tensor core
    if (nchunks > 0) {
      constexpr uint32_t idesc_qk = make_idesc(kFmtE4M3, kFmtE4M3, 0, 0, kM, kN);
      constexpr uint32_t idesc_pv_hi = make_idesc(kFmtE4M3, kFmtE4M3, 0, 1, kM, C::NV);
      constexpr uint32_t idesc_pv_lo = make_idesc(kFmtE5M2, kFmtE4M3, 0, 1, kM, C::NV);
      const uint64_t kdesc0 = make_sdesc(smem_u32(sKV), 16, 1024, kSwizzle128);
      const uint64_t ktail0 = make_sdesc(smem_u32(sKV) + C::NF * C::ATOM, 16, 512, kSwizzle64);
      const uint64_t qdesc0 = make_sdesc(smem_u32(sQ), 16, 1024, kSwizzle128);
      const uint64_t qtail0 = make_sdesc(smem_u32(sQ) + C::QSF * kM * 128, 16, 512, kSwizzle64);
      const uint64_t vdesc0 = make_sdesc(smem_u32(sKV), C::ATOM, 1024, kSwizzle128);
      const uint64_t pdesc0 = make_sdesc(smem_u32(sP), 16, 1024, kSwizzle128);
      const bool leader = elect_one() != 0;
      bool ok = wwait(q_ready, 0);
      if (!ok) fail(4);
      const uint32_t tmem = tmem_base();                 // (q is in it)
      int qk = 0, pv = 0;
      // S = q K^T of chunk qk: both terms of q over the key columns, in steps of 32
      auto issue_qk = [&]() {
        const int rg = qk & 1;
        if (!wwait(&kv_full[rg], (uint32_t)(qk / 2) & 1)) { fail(5); ok = false; return; }
        fence_proxy_async_smem();
        tc_fence_after();
        if (leader) {
          const uint64_t kst = kdesc0 + (uint64_t)((rg * kN * 128) >> 4);
          const uint64_t ktl = ktail0 + (uint64_t)((rg * kN * 64) >> 4);
          const uint32_t dS = tmem + C::SCOL + rg * (kN / 2);
#pragma unroll
          for (int ks = 0; ks < C::KSTEPS; ++ks) {
            const int d = ks * 32;
            const uint32_t acc = ks > 0 ? 1u : 0u;
            if (d < C::NF * 128) {
              const uint64_t bdesc = kst + (uint64_t)(((d / 128) * C::ATOM + (d % 128)) >> 4);
              if (d < C::QT) {
                mma_ws_ts<0>(dS, tmem + C::QCOL + d / 4, bdesc, idesc_qk, acc);
                mma_ws_ts<1>(dS, tmem + C::QCOL + C::QT / 4 + d / 4, bdesc, idesc_qk, 1u);
              } else {
                const int dq = d - C::QT;
                const uint64_t adesc = qdesc0 + (uint64_t)(((dq / 128) * (kM * 128) + (dq % 128)) >> 4);
                mma_ws<0>(dS, adesc, bdesc, idesc_qk, acc);
                mma_ws<1>(dS, adesc + (uint64_t)(C::QPIECE >> 4), bdesc, idesc_qk, 1u);
              }
            } else {
              const int dt = d - C::NF * 128;
              mma_ws<0>(dS, qtail0 + (uint64_t)(dt >> 4), ktl + (uint64_t)(dt >> 4), idesc_qk, acc);
              mma_ws<1>(dS, qtail0 + (uint64_t)((C::QPIECE + dt) >> 4), ktl + (uint64_t)(dt >> 4), idesc_qk, 1u);
            }
          }
          mma_commit(&s_full[rg]);
        }
        __syncwarp();
        ++qk;
      };
      // O += P V of chunk pv; each half of the region is free once its keys are done
      auto issue_pv = [&]() {
        const int rg = pv & 1;
        if (!wwait(&p_full[rg], (uint32_t)(pv / 2) & 1)) { fail(6); ok = false; return; }
        tc_fence_after();
        if (leader) {
          const uint64_t vst = vdesc0 + (uint64_t)((rg * kN * 128) >> 4);
          const uint64_t pst = pdesc0 + (uint64_t)((rg * 2 * C::PTERM) >> 4);
#pragma unroll
          for (int ks = 0; ks < kN / 32; ++ks) {
#pragma unroll
            for (int nv = 0; nv < C::NMMV; ++nv) {
              const uint64_t bdesc = vst + (uint64_t)((nv * (C::NV / 128) * C::ATOM + ks * 32 * 128) >> 4);
              const uint32_t dO = tmem + C::OCOL + nv * (C::NV / 2);
              mma_ws<0>(dO, pst + (uint64_t)((ks * 32) >> 4), bdesc, idesc_pv_hi,
                        (pv > 0 || ks > 0) ? 1u : 0u);
              mma_ws<1>(dO, pst + (uint64_t)((C::PTERM + ks * 32) >> 4), bdesc, idesc_pv_lo, 1u);
            }
            if (ks & 1) mma_commit(&kv_empty[2 * rg + ks / 2]);
          }
        }
        __syncwarp();
        ++pv;
      };
      while (ok && pv < nchunks) {
        issue_qk();
        if (ok && qk < nchunks) issue_qk();
        while (ok && pv < qk) issue_pv();
      }
      if (leader) {
        mma_commit(mma_done);
        mbar_wait(mma_done, 0, p.wait_ns, no_abort);
        // drain: the last arrivals of the commit-fed barriers
        for (int i = max(0, pv - 2); i < pv; ++i)
          for (int u = 0; u < 2; ++u) mbar_wait(&kv_empty[2 * (i & 1) + u], (uint32_t)(i / 2) & 1, p.wait_ns, no_abort);
        for (int i = max(0, qk - 2); i < qk; ++i) mbar_wait(&s_full[i & 1], (uint32_t)(i / 2) & 1, p.wait_ns, no_abort);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax + output
    // lane quarter `quarter` of TMEM: head rows 32 (quarter & 1) + lane, keys
    // 64 (quarter / 2) of a chunk; of those, warp side `c` takes 32
    const int sw = warp - kFirstSoftmax;                 // 0..7
    const int quarter = warp & 3, c = sw >> 2;
    const int r = (quarter & 1) * 32 + lane, kg = quarter >> 1;
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const int h = hs * kM + r;                           // head row of the unit
    const bool head_ok = r < nrows;
    // in a dense call the rows may be of several queries: this row's sees
    // slots up to `last`
    const int last = packed ? Lb - p.T + p.by_H(h) : 0x7fffffff;
    float f_h = 0.f;
    split_q_rows<DK, DV>(q4, 4 * sw, lane, sQ, sP, sE);
    split_q_rows<DK, DV>(q2, 32 + 2 * sw, lane, sQ, sP, sE);
    fence_proxy_async_smem();
    bar_sync(1, 544);                                    // with the gather warps' rows and the TMEM
    const uint32_t tmem = tmem_base();
    if (nchunks > 0) {
      f_h = sE[r];
      if constexpr (C::QT > 0) {
        // this side's term (0: hi, 1: lo) of row r into TMEM, in both lane halves
#pragma unroll
        for (int a = 0; a < C::QT / 128; ++a) {
          uint32_t v[32];
          const uint8_t* src = sP + (c * (C::QT / 128) + a) * (kM * 128) + r * 128;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const uint4 w = *reinterpret_cast<const uint4*>(src + ((x ^ (r & 7)) << 4));
            v[4 * x] = w.x; v[4 * x + 1] = w.y; v[4 * x + 2] = w.z; v[4 * x + 3] = w.w;
          }
          tmem_st32(tmem + lane_addr + C::QCOL + c * (C::QT / 4) + a * 32, v);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    }
    bar_sync(4, 256);                                    // the staged terms are read: the P buffers are free
    float R = -INFINITY, R_top = -INFINITY, l = 0.f;     // l: this thread's keys' share of the row sum
    bool ok = true;
    // a failed wait leaves the loop running without waits: the warps of a
    // barrier all arrive
    for (int j = 0; j < nchunks; ++j) {
      const int pb = j & 1;
      const uint32_t ph = (uint32_t)(j / 2) & 1;
      // 1. 32 scaled logits and their maximum
      if (ok && !wwait(&par_full[pb], ph)) { fail(7); ok = false; }
      // (two keys an instruction where FP32 comes packed; the row's power of two
      // meets the key's scale, while q K^T runs, before it meets the sum, which
      // with 2^102 and more of it would overflow in front of a small scale)
      const ulonglong2* par = reinterpret_cast<const ulonglong2*>(sPar + pb * 3 * kN + kg * 64 + c * 32);
      const uint64_t f2 = pair2(f_h, f_h);
      uint64_t x[16];
      float cm = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const ulonglong2 a = par[i];
        x[2 * i] = mul2(a.x, f2);
        x[2 * i + 1] = mul2(a.y, f2);
      }
      if (ok && !wwait(&s_full[pb], ph)) { fail(8); ok = false; }
      tc_fence_after();
      uint32_t s[32];
      tmem_ld32(tmem + lane_addr + C::SCOL + pb * (kN / 2) + c * 32, s);
      tmem_wait_ld_dep(s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const ulonglong2 lg = par[kN / 4 + i];
        x[2 * i] = fma2(pair2u(s[4 * i], s[4 * i + 1]), x[2 * i], lg.x);
        x[2 * i + 1] = fma2(pair2u(s[4 * i + 2], s[4 * i + 3]), x[2 * i + 1], lg.y);
      }
      const int past = last - (slot0 + j * kN + kg * 64 + c * 32);   // keys i > past are not this row's
      if (__any_sync(0xffffffffu, past < 31)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 y = unpair2(x[i]);
          x[i] = pair2(2 * i > past ? -INFINITY : y.x, 2 * i + 1 > past ? -INFINITY : y.y);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 x0 = unpair2(x[2 * i]), x1 = unpair2(x[2 * i + 1]);
        cm = max3(cm, x0.x, x0.y);
        cm = max3(cm, x1.x, x1.y);
      }
      // 2. the row's maximum over its four threads, and the reference
      float* mx = sMx + pb * 4 * kM + r;
      mx[(kg * 2 + c) * kM] = cm;
      bar_sync(2 + (quarter & 1), 128);
      const float m = fmaxf(fmaxf(mx[0], mx[kM]), fmaxf(mx[2 * kM], mx[3 * kM]));
      float Rn = m > R + kTop ? m - kHead : R;
      if (slot1 - slot0 > kLongPart) {
        if (m < R + (kHead - kDrop) && m != -INFINITY) Rn = fmaxf(m - kHead, R_top - kDepth);
        R_top = fmaxf(R_top, Rn);
      }
      const bool moved = R != -INFINITY && Rn != R;
      const float alpha = moved ? exp2f(R - Rn) : 1.f;
      l *= alpha;
      R = Rn;
      // 3. P in two terms, to shared memory (free: the q K^T of this chunk
      //    came after the P V that read the buffer)
      const float nR = R == -INFINITY ? 0.f : -R;
      const uint64_t nR2 = pair2(nR, nR);
      const ulonglong2* inv = par + 2 * kN / 4;
      uint8_t* prow = sP + pb * 2 * C::PTERM + r * 128;
      uint64_t rs0 = 0ull, rs1 = 0ull;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const ulonglong2 iv = inv[4 * g + i];
          const float2 y0 = unpair2(add2(x[8 * g + 2 * i], nR2)), y1 = unpair2(add2(x[8 * g + 2 * i + 1], nR2));
          const float e0 = ex2_approx(y0.x), e1 = ex2_approx(y0.y), e2 = ex2_approx(y1.x), e3 = ex2_approx(y1.y);
          rs0 = fma2(pair2(e0, e1), iv.x, rs0);
          rs1 = fma2(pair2(e2, e3), iv.y, rs1);
          uint32_t h0, l0, h1, l1;
          split2<__NV_E5M2>(e0, e1, h0, l0);
          split2<__NV_E5M2>(e2, e3, h1, l1);
          hw[i] = h0 | (h1 << 16);
          lw[i] = l0 | (l1 << 16);
        }
        uint8_t* d = prow + (((kg * 4 + c * 2 + g) ^ (r & 7)) << 4);
        *reinterpret_cast<uint4*>(d) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        *reinterpret_cast<uint4*>(d + C::PTERM) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
      }
      const float2 rs = unpair2(add2(rs0, rs1));
      l += rs.x + rs.y;
      fence_proxy_async_smem();
      // 4. the accumulator follows the reference, once the P V before this
      //    chunk is done (that of an even chunk's predecessor is: its q K^T
      //    came after it)
      if (__any_sync(0xffffffffu, moved)) {
        if (ok && (j & 1) && !wwait(&kv_empty[2 * ((j - 1) & 1) + 1], (uint32_t)((j - 1) / 2) & 1)) { fail(10); ok = false; }
        tc_fence_after();
        tmem_scale<C::OCOLS / 2>(tmem + lane_addr + C::OCOL + c * (C::OCOLS / 2), alpha);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&par_empty[pb]);
        mbar_arrive(&p_full[pb]);
      }
    }
    // output: the row's sum over its four threads, then each thread a
    //    quarter of the row's value columns
    float* xl = sMx + (nchunks & 1) * 4 * kM + r;        // read last in chunk nchunks - 2
    xl[(kg * 2 + c) * kM] = l;
    bar_sync(2 + (quarter & 1), 128);
    l = (xl[0] + xl[kM]) + (xl[2 * kM] + xl[3 * kM]);
    if (ok && nchunks > 0 && !wwait(&kv_empty[2 * ((nchunks - 1) & 1) + 1], (uint32_t)((nchunks - 1) / 2) & 1)) {
      fail(12);
      ok = false;
    }
    // A thread has a quarter of one row in 16-byte pieces, which as stores of
    // their own would touch 32 lines an instruction: the warp's 32 quarters
    // are turned in the keys' regions (every MMA is done) and leave as whole
    // 128-byte lines.  The pitch keeps the pieces of eight threads on
    // different banks.  (Bulk copies of the quarters, one a thread, took 2000
    // cycles to issue.)
    constexpr int TC = C::OCOLS / 2;                     // value columns of a thread
    constexpr int PITCH = TC * 2 + 16;
    static_assert(256 * PITCH <= C::KV_BYTES, "output staging");
    // first head row of the unit (and split) in the output or the parts
    const size_t orow = (p.nsplit == 1 ? (size_t)unit : (size_t)unit * p.nsplit + split) * p.HR;
    if (ok && nchunks > 0) {
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : *sUnit / l;    // (a NaN stays one)
      constexpr int W = TC < 32 ? 16 : 32;
      // TMEM column x of the accumulator: MMA x / (NV/2), its columns
      // [kg NV/2, + NV/2) in this lane half; a thread's columns are in one MMA
      static_assert(TC <= C::NV / 2, "a thread's columns lie side by side");
      const int v00 = c * TC / (C::NV / 2) * C::NV + kg * (C::NV / 2) + c * TC % (C::NV / 2);
      uint8_t* mine = sKV + (sw * 32 + lane) * PITCH;
#pragma unroll 1
      for (int x0 = 0; x0 < TC; x0 += W) {
        uint32_t o[W];
        if constexpr (W == 32) tmem_ld32(tmem + lane_addr + C::OCOL + c * TC + x0, o);
        else tmem_ld16(tmem + lane_addr + C::OCOL + c * TC + x0, o);
        tmem_wait_ld_dep(o);
        float f = inv;
        if (p.nsplit > 1) {
          float m4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < W; ++i) m4[i & 3] = fmaxf(m4[i & 3], fabsf(__uint_as_float(o[i])));
          const float mo = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          // the power of two that brings the group's largest into [2^14, 2^15)
          const int e = min(max(127 + 14 - (int)(__float_as_uint(mo * inv) >> 23), -120), 126);
          f = inv * __uint_as_float((uint32_t)(127 + e) << 23);
          if (head_ok) p.part_f[(orow + h) * (DV / W) + (v00 + x0) / W] = __uint_as_float((uint32_t)(127 - e) << 23);
        }
#pragma unroll
        for (int g = 0; g < W / 8; ++g) {
          uint32_t w[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float o0 = __uint_as_float(o[8 * g + 2 * y]) * f, o1 = __uint_as_float(o[8 * g + 2 * y + 1]) * f;
            w[y] = p.nsplit > 1 ? pack_f16x2(o0, o1) : pack_bf16x2(o0, o1);
          }
          *reinterpret_cast<uint4*>(mine + x0 * 2 + 16 * g) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
      constexpr int LPR = TC * 2 / 16;                   // lanes of a quarter row
      uint16_t* base = p.nsplit == 1 ? p.out : reinterpret_cast<uint16_t*>(p.part_o);
      const int r0 = r - lane, lr = lane / LPR, lc = lane % LPR;
#pragma unroll
      for (int i = 0; i < LPR; ++i) {
        const int rr = i * (32 / LPR) + lr;
        const uint4 w = *reinterpret_cast<const uint4*>(sKV + (sw * 32 + rr) * PITCH + lc * 16);
        if (r0 + rr < nrows) *reinterpret_cast<uint4*>(base + (orow + hs * kM + r0 + rr) * DV + v00 + lc * 8) = w;
      }
    }
    if (ok && kg == 0 && c == 0 && head_ok) {
      const float lse2 = l == 0.f ? -INFINITY : R + log2f(l);
      if (p.nsplit == 1) {
        if (p.lse != nullptr) p.lse[orow + h] = lse2 * 0.6931471805599453f;
      } else {
        p.part_lse[orow + h] = lse2;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem_base(), kTmemCols);
  }
}

// Merge the key splits of each head row (H rows to a unit): weights 2^(lse_s - max).  A thread
// takes eight columns of a head and the splits four at a time, with the
// batch's loads issued before the first is used and a running maximum.  128
// threads of up to 80 registers fit beside an attention CTA, so that the
// blocks can wait there for its end.
constexpr int kCombineThreads = 128;
template <int DV>
__global__ void __launch_bounds__(kCombineThreads, 6) attn8_combine_kernel(const __half* part_o, const float* part_f,
                                                                           const float* part_lse, uint16_t* out,
                                                                           float* lse, int heads, int H, int nsplit) {
  constexpr int kBatch = 4, TPH = DV / 8, W = DV >= 128 ? 32 : 16;
  pdl_wait();
  const int gh = blockIdx.x * (kCombineThreads / TPH) + threadIdx.x / TPH;
  if (gh >= heads) return;
  const int row = gh / H, d0 = (threadIdx.x % TPH) * 8;
  // split s of this head lies at first + s H
  const size_t first = (size_t)row * nsplit * H + (gh - row * H);
  const float* pl = part_lse + first;
  const float* pf = part_f + first * (DV / W) + d0 / W;
  const __half* po = part_o + first * DV + d0;
  float mx = -INFINITY, wsum = 0.f, acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int s = nsplit; s > 0; s -= kBatch) {
    float l[kBatch], f[kBatch];
    uint4 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      l[i] = -INFINITY;
      if (i < s) {
        l[i] = *pl;
        f[i] = *pf;
        v[i] = *reinterpret_cast<const uint4*>(po);
        pl += H;
        pf += H * (DV / W);
        po += H * DV;
      }
    }
    // (a NaN part counts as no maximum but is added: the sum becomes NaN)
    const float m = fmaxf(mx, fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])));
    const bool nan = isnan(l[0]) || isnan(l[1]) || isnan(l[2]) || isnan(l[3]);
    if (m == -INFINITY && !nan) continue;
    const float alpha = m == -INFINITY ? 1.f : exp2f(mx - m);
    mx = m;
    wsum *= alpha;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= alpha;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (l[i] == -INFINITY) continue;                     // an empty part's output was never written
      const float w = exp2f(l[i] - mx);
      wsum += w;
      const float wf = w * f[i];
      const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&u[c]));
        acc[2 * c] = fmaf(wf, x.x, acc[2 * c]);
        acc[2 * c + 1] = fmaf(wf, x.y, acc[2 * c + 1]);
      }
    }
  }
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
  *reinterpret_cast<uint4*>(out + (size_t)gh * DV + d0) = make_uint4(w[0], w[1], w[2], w[3]);
  if (d0 == 0 && lse != nullptr) lse[gh] = wsum == 0.f ? -INFINITY : (mx + log2f(wsum)) * 0.6931471805599453f;
}

template <int DK, int DV, bool PAGED>
cudaError_t launch_t(const LaunchCtx& c, const Params& p) {
  using C = Cfg<DK, DV>;
  static std::atomic<int> granted[kMaxDevices];
  cudaError_t e = grant_smem(attn8_kernel<DK, DV, PAGED>, C::BYTES, c.device, granted);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn8_kernel<DK, DV, PAGED>, dim3((unsigned)((long long)p.units * p.nsplit * p.hsplit)), dim3(kThreads),
                 C::BYTES, c.stream, p);
  if (e != cudaSuccess) return e;
  note_launches(1);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.nsplit == 1) return e;
  // a programmatic dependent: its blocks may start while the attention drains
  const int heads = p.units * p.HR;
  const int per = kCombineThreads / (DV / 8);
  e = launch_pdl(attn8_combine_kernel<DV>, dim3((unsigned)((heads + per - 1) / per)), dim3(kCombineThreads), 0, c.stream,
                 (const __half*)p.part_o, (const float*)p.part_f, (const float*)p.part_lse, p.out, p.lse, heads, p.HR,
                 p.nsplit);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Units of a call, the CTAs that share one's head rows, and its key splits:
// one wave of CTAs (one per SM) when there are fewer than SMs, never less than
// one chunk to a split.
struct Plan {
  long long units;
  int HR, hsplit, nsplit;
};
Plan plan(const Attn8Args& a, bool dense, int num_sms) {
  Plan p;
  p.units = dense ? a.B : (long long)a.B * a.T;
  p.HR = dense ? a.T * a.H : a.H;
  p.hsplit = (p.HR + kM - 1) / kM;
  const long long ctas = p.units * p.hsplit, chunks = ((dense ? a.S : a.k) + kN - 1) / kN;
  long long n = num_sms / ctas;
  if (n < 1) n = 1;
  // no more than there are equal shares: of 16 chunks nine splits would take two each
  const long long share = (chunks + n - 1) / n;
  p.nsplit = (int)((chunks + share - 1) / share);
  return p;
}

// FP16 outputs, their factors (at most d_v / 16 a head) and log2-sum-exps
size_t part_bytes(const Plan& p, int d_v) {
  return p.nsplit > 1 ? (size_t)p.units * p.nsplit * p.HR * (d_v * 2 + d_v / 16 * 4 + 4) : 0;
}

}  // namespace

// Workspace of the attention over an 8-bit cache: of a sparse or a dense call,
// and of either.
size_t attn8_call_bytes(const Attn8Args& a, bool dense, int num_sms) {
  return (part_bytes(plan(a, dense, num_sms), a.d_v) + 255) / 256 * 256;
}
size_t attn8_workspace_bytes(const Attn8Args& a, int num_sms) {
  const size_t s = attn8_call_bytes(a, false, num_sms), d = attn8_call_bytes(a, true, num_sms);
  return s > d ? s : d;
}

cudaError_t launch_attn8(const LaunchCtx& c, const Attn8Args& a) {
  Params p = {};
  p.map = a.map;
  p.q = a.q;
  p.kv8 = a.kv8;
  p.kv_scale = a.kv_scale;
  p.idx = a.idx;
  p.dense_rows = a.dense_rows;
  p.out = a.out;
  p.lse = a.lse;
  p.T = a.T;
  p.H = a.H;
  p.k = a.k;
  const Plan pl = plan(a, a.idx == nullptr, c.num_sms);
  p.units = (int)pl.units;
  p.HR = pl.HR;
  p.hsplit = pl.hsplit;
  p.nsplit = pl.nsplit;
  p.by_T = Divisor::of(p.T);
  p.by_H = Divisor::of(p.H);
  p.by_nsplit = Divisor::of(p.nsplit);
  p.by_hsplit = Divisor::of(p.hsplit);
  p.scale_log2 = a.tau * 1.4426950408889634f;
  p.ahead = c.num_sms;
  p.wait_ns = c.wait_ns;
  p.err = c.err;
  if (p.nsplit > 1) {
    if (a.ws == nullptr) return cudaErrorInvalidValue;
    const size_t n = (size_t)pl.units * p.nsplit * p.HR;
    p.part_o = static_cast<__half*>(a.ws);
    p.part_f = reinterpret_cast<float*>(p.part_o + n * a.d_v);
    p.part_lse = p.part_f + n * (a.d_v / 16);
  }
  const bool paged = a.map.page_size != 0;
  if (a.d_k == 576 && a.d_v == 512) return paged ? launch_t<576, 512, true>(c, p) : launch_t<576, 512, false>(c, p);
  if (a.d_k == 80 && a.d_v == 64) return paged ? launch_t<80, 64, true>(c, p) : launch_t<80, 64, false>(c, p);
  return cudaErrorInvalidValue;
}

}  // namespace dsa
