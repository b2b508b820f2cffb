// Sparse and dense MQA/MLA attention over an 8-bit latent cache, on tcgen05.
//
// The cache holds one e4m3 row k8 of d_k bytes and one FP32 scale s per token,
// shared by all heads; the value is the row's first d_v columns.  With
// a = tau log2(e):
//   x_k = a s_k (q . k8_k) + log2 s_k,        R a running reference,
//   P_k = 2^(x_k - R) = 2^(logit_k - R) s_k,  l = sum_k P_k / s_k,
//   out = sum_k P_k k8_k[:d_v] / l,           lse = (R + log2 l) ln 2.
// The token's scale is folded into the exponent, so the cached bytes go to
// the tensor cores as they are, in both products: no dequantised copy of a
// key exists anywhere, a key costs 576 bytes of shared memory instead of
// 1152, and the gather moves half the bytes of the BF16 cache.
//
// kind::f8f6f4 multiplies e4m3 by e4m3 at twice the BF16 rate, so the other
// operand is split in two e4m3 terms and every product runs twice, at the
// cost of one BF16 product:
//   * q = 2^e (q_hi + q_lo), 2^e per head row with max|q| <= 448 * 2^e.  A
//     BF16 number has 8 significant bits and e4m3 four, so the two terms give
//     q exactly down to 2^-10 of the row's largest, and within 2^-19 of it
//     below (e4m3's subnormal step);
//   * P = P_hi + P_lo, rounded to nearest at 2^-9 of P or better (BF16 would
//     be 2^-9).  R is kept so that the largest P of a row lies in [2^6, 2^8]:
//     the subnormal step is then 2^-15 of the largest or less.
// Logits, P before its rounding, l and the output accumulate in FP32.
//
// Work split.  All heads of one query are the MMA M dimension (128 rows).
// A 128 x 512 FP32 accumulator would fill TMEM, so two CTAs share a query,
// one per half of the value columns; few queries also split their keys, and
// a combine kernel merges the parts.
// Per CTA: TMEM holds O (128 x 256) | two S/P buffers of 64 columns | q_hi
// and q_lo of the first 256 key columns.  Shared memory holds the rest of q
// (80 KB) and a ring of four slots of 64 keys (144 KB).
// Warp roles (384 threads): warp 0 issues the MMAs; warp 1 forms the
// per-key constants; warps 2 and 3 gather rows with 16-byte cp.async
// that arrive on the slot's barrier by themselves; warps 4-7 and 8-11 are two
// softmax groups that take the chunks in turn (thread = head row), so a
// group has two chunk periods for its work.  The reference R goes from one
// group to the other through shared memory; it moves only when a chunk's
// maximum exceeds it by 2 (log2 units), and then the accumulator is rescaled
// once, after the P V before it.
#include <cuda_fp8.h>
#include <math.h>

#include "internal.h"
#include "sm100.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kN = 64;                 // keys per chunk
constexpr int kSlots = 4;              // chunks the ring holds
constexpr int kRing = kN * kSlots;     // ring rows
constexpr int kMmaWarp = 0, kParamWarp = 1, kFirstSoftmax = 4;
constexpr int kThreads = 384;         // 12 warps: 168 registers a thread
constexpr uint32_t kTmemCols = 512;
constexpr float kHead = 6.f;           // log2 of the largest P of a row when R is set
constexpr float kSlack = 2.f;          // how far a maximum may pass before R moves (2^(6+2) < 448)

template <int DK, int DV>
struct Cfg {
  static constexpr int KSTEPS = (DK + 31) / 32;        // 32-byte MMA K steps
  static constexpr int NF = DK >= 128 ? DK / 128 : 1;  // 128-byte atoms of a row
  static constexpr int TAIL = DK > NF * 128 ? 1 : 0;   // one 64-byte atom more
  static constexpr int NHALF = DV >= 128 ? 2 : 1;
  static constexpr int DVH = DV / NHALF;
  static constexpr uint32_t OCOL = 0;
  static constexpr uint32_t SCOL = DVH;
  static constexpr uint32_t QCOL = SCOL + 2 * kN;
  // leading key columns whose q lies in TMEM (whole atoms)
  static constexpr int QT = (int)(kTmemCols - QCOL) / 2 * 4 / 128 * 128 >= DK ? 0 : (int)(kTmemCols - QCOL) / 2 * 4 / 128 * 128;
  static constexpr int QSF = NF - QT / 128;            // q atoms in shared memory
  static constexpr int QPIECE = QSF * 128 * 128 + TAIL * 128 * 64;
  static constexpr int ATOM = kRing * 128;             // bytes of one ring atom
  static constexpr int RING_BYTES = NF * ATOM + TAIL * kRing * 64;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * QPIECE;
  static constexpr int OFF_PAR = OFF_KV + RING_BYTES;  // [2][64] {a s, log2 s}, [2][64] 1 / s
  static constexpr int OFF_M = OFF_PAR + 2 * kN * 12;  // [128] the running reference
  static constexpr int OFF_BAR = OFF_M + 128 * 4;
  static constexpr int NBARS = 1 + 2 * kSlots + 2 + 2 + 2 + 2 + 1 + 8;
  static constexpr int OFF_MISC = OFF_BAR + NBARS * 8;
  static constexpr int BYTES = OFF_MISC + 16;
  static_assert(BYTES <= 232448, "shared memory per CTA");
  static_assert(OFF_KV % 1024 == 0 && OFF_BAR % 8 == 0, "alignment");
  static_assert(QCOL + 2 * (QT / 4) <= kTmemCols, "TMEM");
  // q's bytes on their way to TMEM pass through the ring's upper half
  static_assert(QT == 0 || (2 * QT * 128 <= 2 * 128 * 128 * 2), "staging");
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
  float* part_o;         // [rows, nsplit, H, d_v] (nsplit > 1), normalised by the part's own l
  float* part_lse;       // [rows, nsplit, H], log2 units
  int T, H, k;
  int rows, nsplit;
  float scale_log2;      // tau log2(e)
  long long wait_ns;
  DevErr* err;
};

__device__ __forceinline__ int pow2_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -100);
}
__device__ __forceinline__ uint32_t e4m3x2_of_half2(__half2 h) {
  return (uint32_t)__nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<__half2_raw*>(&h), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 half2_of_e4m3x2(uint32_t v) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)v, __NV_E4M3));
}
// two e4m3 terms of a pair of numbers (|a|, |b| <= 448): low 16 bits of hi, lo
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  hi = e4m3x2_of_half2(h);
  lo = e4m3x2_of_half2(__hsub2(h, half2_of_e4m3x2(hi)));
}

__device__ __forceinline__ void mma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <int DK, int DV, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) attn8_kernel(Params p) {
  using C = Cfg<DK, DV>;
  extern __shared__ uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    // self-check: the swizzled layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) report_error(p.err, DSA_ERR_DEVICE_BOUNDS, ERR_SITE_ATTN8 | (0xAu << 8));
    return;
  }
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sKV = smem + C::OFF_KV;
  float2* sPar = reinterpret_cast<float2*>(smem + C::OFF_PAR);        // [2][64]
  float* sInv = reinterpret_cast<float*>(smem + C::OFF_PAR + 2 * kN * 8);
  float* sM = reinterpret_cast<float*>(smem + C::OFF_M);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_ready = bars;                    // q in shared memory and TMEM (8 softmax warps)
  uint64_t* kv_full = q_ready + 1;             // [slot] rows landed (2 gather warps, every lane)
  uint64_t* kv_empty = kv_full + kSlots;       // [slot] P V of the slot's chunk complete (commit)
  uint64_t* par_full = kv_empty + kSlots;      // [2] per-key constants written (32 lanes)
  uint64_t* par_empty = par_full + 2;          // [2] and read (4 warps)
  uint64_t* s_full = par_empty + 2;            // [2] Q K^T complete (commit)
  uint64_t* p_full = s_full + 2;               // [2] P written (4 warps)
  uint64_t* mma_done = p_full + 2;
  uint64_t* m_bar = mma_done + 1;              // [2 groups][4 quarters] reference published
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = blockIdx.x % C::NHALF;
  const int rest = blockIdx.x / C::NHALF;
  const int row = rest / p.nsplit;             // b * T + t
  const int split = rest - row * p.nsplit;
  const int b = row / p.T, t = row - b * p.T;
  const int Lb = p.map.len(b, threadIdx.x == 0 ? p.err : nullptr, ERR_SITE_ATTN8);
  const bool dense = p.idx == nullptr || t < p.dense_rows;
  const int nslots = dense ? Lb - p.T + t + 1 : p.k;      // slots of this row
  // an equal share of the row's chunks for every split
  const int kc = ((nslots + kN - 1) / kN + p.nsplit - 1) / p.nsplit * kN;
  const int slot0 = min(split * kc, nslots), slot1 = min(slot0 + kc, nslots);
  const int nchunks = (slot1 - slot0 + kN - 1) / kN;

  if (threadIdx.x == 0) {
    mbar_init(q_ready, 8);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&kv_full[i], 64);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&par_full[i], 32);
      mbar_init(&par_empty[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
    }
    mbar_init(mma_done, 1);
    for (int i = 0; i < 8; ++i) mbar_init(&m_bar[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if constexpr (DK % 128 != 0 && C::TAIL == 0) {
    // columns DK.. of the ring's atom meet zero columns of q in the last K
    // step: they must not hold NaN bytes
    for (int i = threadIdx.x; i < kRing * 8; i += kThreads)
      if (i % 8 >= DK / 16) *reinterpret_cast<uint4*>(sKV + (i / 8) * 128 + (((i % 8) ^ ((i / 8) & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

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
  const int32_t* irow = dense ? nullptr : p.idx + (size_t)row * p.k;
  // index of slot s of this split; -1 past the end, for an empty slot and for
  // an index outside [0, L_b)
  auto load_idx = [&](int s) -> int { return s < slot1 ? (dense ? s : irow[s]) : -1; };
  // cache row (relative to the sequence's first in a contiguous cache) or -1
  auto row_of = [&](int v) -> int {
    if (v < 0 || v >= Lb) return -1;
    return PAGED ? (int)p.map.row<true>(b, v) : v;
  };
  const long long base_row = PAGED ? 0 : (long long)b * p.map.S;

  if (warp == 2 || warp == 3) {
    // ------------------------------------------------------------ gather
    // warp g copies keys [32 g, 32 g + 32) of every chunk
    const int g = warp - 2;
    const uint8_t* base = p.kv8 + base_row * DK;
    const int kl = 32 * g + lane;
    int r_cur = row_of(load_idx(slot0 + kl));
    int i_next = load_idx(slot0 + kN + kl);
    bool ok = true;
    for (int j = 0; j < nchunks; ++j) {
      const int st = j % kSlots;
      if (j >= kSlots && !wwait(&kv_empty[st], (uint32_t)(j / kSlots - 1) & 1)) { fail(1); ok = false; break; }
      // q's bytes pass through slots 2 and 3 on their way to TMEM
      if (C::QT > 0 && (j == 2 || j == 3) && !wwait(q_ready, 0)) { fail(2); ok = false; break; }
      const int r_next = row_of(i_next);
      i_next = load_idx(slot0 + (j + 2) * kN + kl);
      uint8_t* dst0 = sKV + (st * kN + 32 * g) * 128;
      const int c = lane & 7, rg = lane >> 3;
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        const int kr = 4 * m + rg;                       // key within the warp's 32
        const int r = __shfl_sync(0xffffffffu, r_cur, kr);
        const uint8_t* src = base + (size_t)(r < 0 ? 0 : r) * DK + c * 16;
        uint8_t* dst = dst0 + kr * 128 + ((c ^ (kr & 7)) << 4);
#pragma unroll
        for (int a = 0; a < C::NF; ++a)
          if (a * 128 + c * 16 < DK) cp_async16_zfill(dst + a * C::ATOM, src + a * 128, r < 0 ? 0u : 16u);
      }
      if constexpr (C::TAIL != 0) {
        const int c4 = lane & 3, rg8 = lane >> 2;
        uint8_t* tail0 = sKV + C::NF * C::ATOM + (st * kN + 32 * g) * 64;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int kr = 8 * m + rg8;
          const int r = __shfl_sync(0xffffffffu, r_cur, kr);
          cp_async16_zfill(tail0 + kr * 64 + ((c4 ^ ((kr >> 1) & 3)) << 4),
                           base + (size_t)(r < 0 ? 0 : r) * DK + C::NF * 128 + c4 * 16, r < 0 ? 0u : 16u);
        }
      }
      cp_async_arrive(&kv_full[st]);
      r_cur = r_next;
    }
    (void)ok;
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == kParamWarp) {
    // ------------------------------------------------------------ per-key constants
    // lane l holds keys l and l + 32 of a chunk
    auto scale_of = [&](int r) -> float { return r < 0 ? 0.f : __ldg(p.kv_scale + base_row + r); };
    auto checked_row = [&](int v) -> int {
      if (v >= Lb) {
        if (half == 0) report_error(p.err, DSA_ERR_DEVICE_BOUNDS, ERR_SITE_ATTN8);
        return -1;
      }
      const int r = row_of(v);
      if (PAGED && v >= 0 && r < 0 && half == 0) report_error(p.err, DSA_ERR_DEVICE_BOUNDS, ERR_SITE_ATTN8 | (1u << 8));
      return r;
    };
    int i_next[2];
    float s_cur[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s_cur[u] = scale_of(checked_row(load_idx(slot0 + lane + 32 * u)));
      i_next[u] = load_idx(slot0 + kN + lane + 32 * u);
    }
    for (int j = 0; j < nchunks; ++j) {
      float s_next[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        s_next[u] = scale_of(checked_row(i_next[u]));
        i_next[u] = load_idx(slot0 + (j + 2) * kN + lane + 32 * u);
      }
      const int pb = j & 1;
      if (j >= 2 && !wwait(&par_empty[pb], (uint32_t)(j / 2 - 1) & 1)) { fail(3); break; }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float s = s_cur[u];
        const bool on = s > 0.f;
        sPar[pb * kN + lane + 32 * u] = make_float2(p.scale_log2 * s, on ? log2f(s) : -INFINITY);
        sInv[pb * kN + lane + 32 * u] = on ? 1.f / s : 0.f;
        s_cur[u] = s_next[u];
      }
      mbar_arrive(&par_full[pb]);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    if (lane == 0 && nchunks > 0) {
      constexpr uint32_t idesc_qk = make_idesc(kFmtE4M3, kFmtE4M3, 0, 0, 128, kN);
      constexpr uint32_t idesc_pv = make_idesc(kFmtE4M3, kFmtE4M3, 0, 1, 128, C::DVH);
      const uint64_t kdesc0 = make_sdesc(smem_u32(sKV), 16, 1024, kSwizzle128);
      const uint64_t ktail0 = make_sdesc(smem_u32(sKV) + C::NF * C::ATOM, 16, 512, kSwizzle64);
      const uint64_t qdesc0 = make_sdesc(smem_u32(sQ), 16, 1024, kSwizzle128);
      const uint64_t qtail0 = make_sdesc(smem_u32(sQ) + C::QSF * 128 * 128, 16, 512, kSwizzle64);
      const uint64_t vdesc0 = make_sdesc(smem_u32(sKV) + (uint32_t)(half * (C::DVH / 128)) * C::ATOM, C::ATOM, 1024,
                                         kSwizzle128);
      bool ok = mbar_wait(q_ready, 0, p.wait_ns, ab);
      if (!ok) fail(4);
      tc_fence_after();
      int qk = 0, pv = 0;
      // S(j) = q K^T: both terms of q over the key columns in steps of 32
      auto issue_qk = [&]() -> bool {
        const int st = qk % kSlots, sb = qk & 1;
        if (!mbar_wait(&kv_full[st], (uint32_t)(qk / kSlots) & 1, p.wait_ns, ab)) { fail(5); return false; }
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t kst = kdesc0 + (uint64_t)((st * kN * 128) >> 4);
        const uint64_t ktl = ktail0 + (uint64_t)((st * kN * 64) >> 4);
        const uint32_t dS = tmem + C::SCOL + sb * kN;
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int ks = 0; ks < C::KSTEPS; ++ks) {
            const int d = ks * 32;
            const uint32_t acc = (term > 0 || ks > 0) ? 1u : 0u;
            if (d < C::NF * 128) {
              const uint64_t bdesc = kst + (uint64_t)(((d / 128) * C::ATOM + (d % 128)) >> 4);
              if (d < C::QT) {
                mma_f8_ts(dS, tmem + C::QCOL + term * (C::QT / 4) + d / 4, bdesc, idesc_qk, acc);
              } else {
                const int dq = d - C::QT;
                mma_f8(dS, qdesc0 + (uint64_t)((term * C::QPIECE + (dq / 128) * 16384 + (dq % 128)) >> 4), bdesc,
                       idesc_qk, acc);
              }
            } else {
              const int dt = d - C::NF * 128;
              mma_f8(dS, qtail0 + (uint64_t)((term * C::QPIECE + dt) >> 4), ktl + (uint64_t)(dt >> 4), idesc_qk, acc);
            }
          }
        mma_commit(&s_full[sb]);
        ++qk;
        return true;
      };
      ok = ok && issue_qk();
      while (ok && pv < nchunks) {
        // Q K^T of the next chunk goes ahead of this chunk's P V, over the
        // S/P buffer of the P V before it: the tensor core takes the MMAs of
        // one thread in the order of their issue
        if (qk < nchunks && !issue_qk()) { ok = false; break; }
        const int st = pv % kSlots, sb = pv & 1;
        if (!mbar_wait(&p_full[sb], (uint32_t)(pv / 2) & 1, p.wait_ns, ab)) { fail(6); ok = false; break; }
        tc_fence_after();
        const uint64_t vst = vdesc0 + (uint64_t)((st * kN * 128) >> 4);
#pragma unroll
        for (int ks = 0; ks < kN / 32; ++ks)
#pragma unroll
          for (int term = 0; term < 2; ++term)
            mma_f8_ts(tmem + C::OCOL, tmem + C::SCOL + sb * kN + term * (kN / 4) + ks * 8,
                      vst + (uint64_t)((ks * 32 * 128) >> 4), idesc_pv, (pv > 0 || ks > 0 || term > 0) ? 1u : 0u);
        mma_commit(&kv_empty[st]);
        ++pv;
      }
      mma_commit(mma_done);
      mbar_wait(mma_done, 0, p.wait_ns, no_abort);
      // drain: the last arrivals of the commit-fed barriers
      for (int i = max(0, pv - kSlots); i < pv; ++i)
        mbar_wait(&kv_empty[i % kSlots], (uint32_t)(i / kSlots) & 1, p.wait_ns, no_abort);
      for (int i = max(0, qk - 2); i < qk; ++i) mbar_wait(&s_full[i & 1], (uint32_t)(i / 2) & 1, p.wait_ns, no_abort);
    }
  } else {
    // ------------------------------------------------------------ softmax + output
    const int grp = (warp - kFirstSoftmax) >> 2, quarter = warp & 3;
    const int h = quarter * 32 + lane;                   // head row == TMEM lane
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const bool head_ok = h < p.H;
    uint8_t* stage = sKV + 2 * kN * 128;                 // ring slots 2 and 3 of each atom
    float f_h = 0.f;
    if (nchunks > 0) {
      // q rows: a warp takes a row at a time, 16 rows; the row's exponent from
      // its maximum, then the two terms of eight columns per lane and step
      constexpr int QV = (DK + 255) / 256;               // 8-column vectors per lane
      const int sw = warp - kFirstSoftmax;
      for (int i = 0; i < 16; ++i) {
        const int hr = sw * 16 + i;
        uint4 v[QV];
        float amax = 0.f;
#pragma unroll
        for (int u = 0; u < QV; ++u) {
          const int col = (u * 32 + lane) * 8;
          v[u] = make_uint4(0u, 0u, 0u, 0u);
          if (hr < p.H && col < DK) v[u] = *reinterpret_cast<const uint4*>(p.q + ((size_t)row * p.H + hr) * DK + col);
          const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
          for (int x = 0; x < 4; ++x)
            amax = fmaxf(amax, fmaxf(__uint_as_float((w[x] & 0x7fffu) << 16), __uint_as_float(w[x] & 0x7fff0000u)));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        const int e = pow2_exponent(amax);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        if (lane == 0) sM[hr] = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int u = 0; u < QV; ++u) {
          const int col = (u * 32 + lane) * 8;
          if (col >= C::NF * 128 + C::TAIL * 64) continue;   // columns DK.. of the last atom are written as zeros
          const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            split2(__uint_as_float(w[x] << 16) * inv, __uint_as_float(w[x] & 0xffff0000u) * inv, hi[x], lo[x]);
          const uint2 H = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
          const uint2 L = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
          const int c16 = (col % 128) / 16, sub = col % 16;
          if (col < C::QT) {
            // staged [atom][128 rows x 128 bytes], hi in the ring's atoms 0, 1, lo in 2, 3
            uint8_t* d = stage + (col / 128) * C::ATOM + hr * 128 + ((c16 ^ (hr & 7)) << 4) + sub;
            *reinterpret_cast<uint2*>(d) = H;
            *reinterpret_cast<uint2*>(d + (C::QT / 128) * C::ATOM) = L;
          } else if (col < C::NF * 128) {
            uint8_t* d = sQ + ((col - C::QT) / 128) * 16384 + hr * 128 + ((c16 ^ (hr & 7)) << 4) + sub;
            *reinterpret_cast<uint2*>(d) = H;
            *reinterpret_cast<uint2*>(d + C::QPIECE) = L;
          } else {
            const int ct = (col - C::NF * 128) / 16;
            uint8_t* d = sQ + C::QSF * 16384 + hr * 64 + ((ct ^ ((hr >> 1) & 3)) << 4) + sub;
            *reinterpret_cast<uint2*>(d) = H;
            *reinterpret_cast<uint2*>(d + C::QPIECE) = L;
          }
        }
      }
    }
    softmax_sync();
    if (nchunks > 0) {
      f_h = sM[h];
      if constexpr (C::QT > 0) {
        // this group's term (0: hi, 1: lo) of row h into TMEM
#pragma unroll
        for (int a = 0; a < C::QT / 128; ++a) {
          uint32_t v[32];
          const uint8_t* src = stage + (grp * (C::QT / 128) + a) * C::ATOM + h * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + ((c ^ (h & 7)) << 4));
            v[4 * c] = x.x; v[4 * c + 1] = x.y; v[4 * c + 2] = x.z; v[4 * c + 3] = x.w;
          }
          tmem_st32(tmem + lane_addr + C::QCOL + grp * (C::QT / 4) + a * 32, v);
        }
        tmem_wait_st();
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    }
    softmax_sync();                                      // sM is read: it holds the reference from here on
    float R = -INFINITY, l = 0.f;                        // l: this group's chunks' share of the row sum
    bool ok = true;
    for (int j = grp; j < nchunks; j += 2) {
      const uint32_t ph = (uint32_t)(j / 2) & 1;
      // 1. the chunk's 64 scaled logits and their maximum
      if (!wwait(&par_full[grp], ph)) { fail(7); ok = false; break; }
      if (!wwait(&s_full[grp], ph)) { fail(8); ok = false; break; }
      tc_fence_after();
      const uint32_t saddr = tmem + lane_addr + C::SCOL + grp * kN;
      uint32_t s0[32], s1[32];
      tmem_ld32(saddr, s0);
      tmem_ld32(saddr + 32, s1);
      tmem_wait_ld_dep(s0);
      tmem_wait_ld_dep(s1);
      const float2* par = sPar + grp * kN;
      const float* inv = sInv + grp * kN;
      float cm = -INFINITY;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float2 a0 = par[i], a1 = par[32 + i];
        const float x0 = fmaf(__uint_as_float(s0[i]) * f_h, a0.x, a0.y);
        const float x1 = fmaf(__uint_as_float(s1[i]) * f_h, a1.x, a1.y);
        s0[i] = __float_as_uint(x0);
        s1[i] = __float_as_uint(x1);
        cm = fmaxf(cm, fmaxf(x0, x1));
      }
      // 2. the reference after the chunk before this one, and after this one
      float Rp = -INFINITY;
      if (j > 0) {
        if (!wwait(&m_bar[(grp ^ 1) * 4 + quarter], (uint32_t)((j - 1) / 2) & 1)) { fail(9); ok = false; break; }
        Rp = sM[h];
      }
      float Rn = Rp;
      if (Rp == -INFINITY) {
        if (cm != -INFINITY) Rn = cm - kHead;
      } else if (cm - kHead > Rp + kSlack) {
        Rn = cm - kHead;
      }
      sM[h] = Rn;
      __syncwarp();
      if (lane == 0) mbar_arrive(&m_bar[grp * 4 + quarter]);
      const bool moved = Rp != -INFINITY && Rn != Rp;
      if (R != Rn) {
        l = R == -INFINITY ? 0.f : l * exp2f(R - Rn);
        R = Rn;
      }
      // 3. the accumulator follows, once the P V before this chunk has landed
      if (__any_sync(0xffffffffu, moved)) {
        if (!wwait(&kv_empty[(j - 1) % kSlots], (uint32_t)((j - 1) / kSlots) & 1)) { fail(10); ok = false; break; }
        tc_fence_after();
        const float alpha = moved ? exp2f(Rp - Rn) : 1.f;
        for (int c = 0; c < C::DVH / 32; ++c) {
          uint32_t o[32];
          const uint32_t oaddr = tmem + lane_addr + C::OCOL + c * 32;
          tmem_ld32(oaddr, o);
          tmem_wait_ld_dep(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(oaddr, o);
        }
        tmem_wait_st();
      }
      // 4. P in two terms: columns [0, 16) hi, [16, 32) lo of the S buffer
      const float nR = Rn == -INFINITY ? 0.f : -Rn;
      uint32_t pk[32];
      float rs0 = 0.f, rs1 = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int k0 = 4 * i + 2 * u;
          const float x0 = __uint_as_float(k0 < 32 ? s0[k0 & 31] : s1[k0 & 31]);
          const float x1 = __uint_as_float(k0 < 32 ? s0[(k0 + 1) & 31] : s1[(k0 + 1) & 31]);
          const float e0 = ex2_approx(x0 + nR), e1 = ex2_approx(x1 + nR);
          rs0 = fmaf(e0, inv[k0], rs0);
          rs1 = fmaf(e1, inv[k0 + 1], rs1);
          split2(e0, e1, hi[u], lo[u]);
        }
        pk[i] = hi[0] | (hi[1] << 16);
        pk[16 + i] = lo[0] | (lo[1] << 16);
      }
      l += rs0 + rs1;
      tmem_st32(saddr, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&par_empty[grp]);
        mbar_arrive(&p_full[grp]);
      }
    }
    // 5. output: both groups' sums at the last reference, then each group
    //    writes half of this CTA's value columns
    float Rl = -INFINITY;
    if (ok && nchunks > 0) {
      const int last = nchunks - 1;
      if ((last & 1) != grp && !wwait(&m_bar[(last & 1) * 4 + quarter], (uint32_t)(last / 2) & 1)) {
        fail(11);
        ok = false;
      }
      if (ok && !wwait(&kv_empty[last % kSlots], (uint32_t)(last / kSlots) & 1)) {
        fail(12);
        ok = false;
      }
      if (ok) {
        tc_fence_after();
        Rl = sM[h];
        if (R != Rl) l = R == -INFINITY ? 0.f : l * exp2f(R - Rl);
      }
    }
    float* xl = reinterpret_cast<float*>(sKV);           // the ring is no longer read
    softmax_sync();
    if (ok && nchunks > 0) xl[grp * 128 + h] = l;
    softmax_sync();
    if (ok && nchunks > 0) l += xl[(grp ^ 1) * 128 + h];
    if (ok) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const float lse2 = l > 0.f ? Rl + log2f(l) : -INFINITY;
      constexpr int OH = C::DVH / 2;                     // value columns per group
      const size_t orow = p.nsplit == 1 ? (size_t)row : (size_t)row * p.nsplit + split;
      if (nchunks > 0) {
        const int v0 = half * C::DVH + grp * OH;
#pragma unroll 1
        for (int c = 0; c < OH / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tmem + lane_addr + C::OCOL + grp * OH + c * 32, o);
          tmem_wait_ld_dep(o);
          if (head_ok && p.nsplit == 1) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + (orow * p.H + h) * DV + v0 + c * 32);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                w[x] = pack_bf16x2(__uint_as_float(o[8 * g + 2 * x]) * inv, __uint_as_float(o[8 * g + 2 * x + 1]) * inv);
              dst[g] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (head_ok) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + (orow * p.H + h) * DV + v0 + c * 32);
#pragma unroll
            for (int g = 0; g < 8; ++g)
              dst[g] = make_float4(__uint_as_float(o[4 * g]) * inv, __uint_as_float(o[4 * g + 1]) * inv,
                                   __uint_as_float(o[4 * g + 2]) * inv, __uint_as_float(o[4 * g + 3]) * inv);
          }
          __syncwarp();
        }
      }
      if (half == 0 && grp == 0 && head_ok) {
        if (p.nsplit == 1) {
          if (p.lse != nullptr) p.lse[orow * p.H + h] = lse2 * 0.6931471805599453f;
        } else {
          p.part_lse[orow * p.H + h] = lse2;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge the key splits of each (row, head): weights 2^(lse_s - max).
template <int DV>
__global__ void __launch_bounds__(DV / 4) attn8_combine_kernel(const float* part_o, const float* part_lse,
                                                               uint16_t* out, float* lse, int H, int nsplit) {
  const size_t row = blockIdx.x / H;
  const int h = blockIdx.x % H;
  const float* ls = part_lse + row * nsplit * H + h;
  const float* po = part_o + (row * nsplit * H + h) * DV + threadIdx.x * 4;
  float mx = -INFINITY;
  for (int s = 0; s < nsplit; ++s) mx = fmaxf(mx, ls[(size_t)s * H]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float wsum = 0.f;
  if (mx != -INFINITY) {
    for (int s = 0; s < nsplit; ++s) {
      const float l = ls[(size_t)s * H];
      if (l == -INFINITY) continue;                      // an empty part's output was never written
      const float w = exp2f(l - mx);
      const float4 v = *reinterpret_cast<const float4*>(po + (size_t)s * H * DV);
      wsum += w;
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
  }
  const float inv = wsum > 0.f ? 1.f / wsum : 0.f;
  *reinterpret_cast<uint2*>(out + (row * H + h) * DV + threadIdx.x * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (threadIdx.x == 0 && lse != nullptr)
    lse[row * H + h] = wsum > 0.f ? (mx + log2f(wsum)) * 0.6931471805599453f : -INFINITY;
}

template <int DK, int DV, bool PAGED>
cudaError_t launch_t(const LaunchCtx& c, const Params& p) {
  using C = Cfg<DK, DV>;
  cudaError_t e = cudaFuncSetAttribute(attn8_kernel<DK, DV, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
  if (e != cudaSuccess) return e;
  attn8_kernel<DK, DV, PAGED><<<(unsigned)((long long)p.rows * p.nsplit * C::NHALF), kThreads, C::BYTES, c.stream>>>(p);
  note_launches(1);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.nsplit == 1) return e;
  attn8_combine_kernel<DV><<<(unsigned)((long long)p.rows * p.H), DV / 4, 0, c.stream>>>(p.part_o, p.part_lse, p.out,
                                                                                       p.lse, p.H, p.nsplit);
  note_launches(1);
  return cudaGetLastError();
}

// Key splits per query row: one wave of CTAs (one per SM) when there are
// fewer rows than SMs, never less than one chunk to a split.
int choose_nsplit(long long rows, int d_v, long long slots, int num_sms) {
  const long long ctas = rows * (d_v >= 128 ? 2 : 1);
  const long long chunks = (slots + kN - 1) / kN;
  long long n = num_sms / ctas;
  if (n < 1) n = 1;
  return (int)(n < chunks ? n : chunks);
}

size_t part_bytes(long long rows, int H, int d_v, int nsplit) {
  return nsplit > 1 ? (size_t)rows * nsplit * H * (d_v + 1) * sizeof(float) : 0;
}

}  // namespace

// Workspace of the attention over an 8-bit cache, for sparse and dense calls.
size_t attn8_workspace_bytes(const Attn8Args& a, int num_sms) {
  const long long rows = (long long)a.B * a.T;
  const size_t s = part_bytes(rows, a.H, a.d_v, choose_nsplit(rows, a.d_v, a.k, num_sms));
  const size_t d = part_bytes(rows, a.H, a.d_v, choose_nsplit(rows, a.d_v, a.S, num_sms));
  return ((s > d ? s : d) + 255) / 256 * 256;
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
  const long long rows = (long long)a.B * a.T;
  p.rows = (int)rows;
  p.nsplit = choose_nsplit(rows, a.d_v, a.idx != nullptr ? a.k : a.S, c.num_sms);
  p.scale_log2 = a.tau * 1.4426950408889634f;
  p.wait_ns = c.wait_ns;
  p.err = c.err;
  if (p.nsplit > 1) {
    if (a.ws == nullptr) return cudaErrorInvalidValue;
    p.part_o = static_cast<float*>(a.ws);
    p.part_lse = p.part_o + (size_t)rows * p.nsplit * a.H * a.d_v;
  }
  const bool paged = a.map.page_size != 0;
  if (a.d_k == 576 && a.d_v == 512) return paged ? launch_t<576, 512, true>(c, p) : launch_t<576, 512, false>(c, p);
  if (a.d_k == 80 && a.d_v == 64) return paged ? launch_t<80, 64, true>(c, p) : launch_t<80, 64, false>(c, p);
  return cudaErrorInvalidValue;
}

}  // namespace dsa
