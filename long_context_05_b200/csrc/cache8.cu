// The 8-bit caches: quantising new rows as they are written to their places,
// and reading ranges back.
//
// A row x of d columns becomes e4m3 bytes and one FP32 scale 2^e:
//   e = the smallest exponent >= -48 with max|x| <= 448 * 2^e,
//   byte_c = e4m3(x_c * 2^-e), rounded to nearest even.
// The scale is a power of two so that x * 2^-e is exact: the one rounding is
// e4m3's own, and a byte times its scale is again exact in BF16, so reading
// back loses nothing.  It costs less than an octave of e4m3's 15 (values down
// to 2^-15 of the row's largest keep their three mantissa bits).  The bound
// on e keeps the scale of a zero row positive; at the other end values past
// 240 * 2^120 are stored as that, so that what a byte stands for is finite.  A
// scale per token is the finest block of tokens and the only one an append can
// write without quantising rows again that were written before.
//
// Both directions are bound by HBM (3 bytes per element).  A row is held in
// the registers of eight lanes (16-byte loads, 8-byte stores or the reverse;
// 64 and 128 contiguous bytes per row and instruction), its maximum taken by
// three shuffles.  One launch serves the attention rows, the indexer's keys
// and the indexer's queries: a decode step appends a few KB, where a launch
// costs more than the work.  The kernels are programmatic dependents of what
// is before them on the stream, so that their launch overlaps its end.
//
// Measured: an 8K prefill's rows (8192 of 576 columns, of 128, and 64 queries
// of 128 each; 221 MB) 37.9 us, 5.8 TB/s; four 32K prefixes read back (278 MB)
// 46.6 us, 6.0 TB/s.  The appends of a decode step take 2.4 us on the device,
// a launch's own time, and 10 us of a host that waits for nothing else.
#include <cuda_fp8.h>

#include "internal.h"
#include "sm100.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 128;
constexpr int kLanes = 8;                          // lanes per row
constexpr int kRows = kThreads / kLanes;           // rows per block and step
constexpr int kQRows = 4;                          // index query rows of a group in flight (short rows, many of them)
constexpr int kMinExp = -48;

__device__ __forceinline__ float max_abs8(const uint4& v) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = fmaxf(m, fmaxf(__uint_as_float((u[i] & 0x7fffu) << 16), __uint_as_float(u[i] & 0x7fff0000u)));
  return m;
}

__device__ __forceinline__ int row_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  // amax = m 2^x with m in [1, 2); 448 = 1.75 * 2^8
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, kMinExp);
}

// both BF16 halves at most 0x7F70 (1.875 * 2^127) in magnitude; NaN stays
__device__ __forceinline__ uint32_t clamp2(uint32_t u) {
  uint32_t lo = u & 0x7fffu, hi = (u >> 16) & 0x7fffu;
  if (lo > 0x7f70u && lo <= 0x7f80u) lo = 0x7f70u;
  if (hi > 0x7f70u && hi <= 0x7f80u) hi = 0x7f70u;
  return (u & 0x80008000u) | lo | (hi << 16);
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// R rows of D columns by eight lanes, V vectors of eight columns each; row i
// lies at src[i] (null: none).  Every load is issued before the first is used.
template <int V, int R>
__device__ __forceinline__ void quantise_rows(const uint16_t* const (&src)[R], int D, uint8_t* const (&dst)[R],
                                              float* const (&scale)[R], int gl) {
  uint4 v[R][V];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * kLanes + gl) * 8;
      v[i][j] = make_uint4(0u, 0u, 0u, 0u);
      if (src[i] != nullptr && col < D) v[i][j] = *reinterpret_cast<const uint4*>(src[i] + col);
    }
  float amax[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    amax[i] = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) amax[i] = fmaxf(amax[i], max_abs8(v[i][j]));
  }
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1)
#pragma unroll
    for (int i = 0; i < R; ++i) amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], d));
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (src[i] == nullptr) continue;
    const int e = min(row_exponent(amax[i]), 120);
    if (e == 120) {
      // 2^120 times a byte past 240 is 2^128, not an FP32 number: such values
      // (1.875 * 2^127 and up) are stored as 240, so that the row stays finite
#pragma unroll
      for (int j = 0; j < V; ++j)
        v[i][j] = make_uint4(clamp2(v[i][j].x), clamp2(v[i][j].y), clamp2(v[i][j].z), clamp2(v[i][j].w));
    }
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * kLanes + gl) * 8;
      if (col >= D) continue;
      const uint32_t u[4] = {v[i][j].x, v[i][j].y, v[i][j].z, v[i][j].w};
      uint32_t q[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        q[x] = e4m3x2(__uint_as_float(u[x] << 16) * inv, __uint_as_float(u[x] & 0xffff0000u) * inv);
      *reinterpret_cast<uint2*>(dst[i] + col) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
    }
    if (gl == 0) *scale[i] = __uint_as_float((uint32_t)(127 + e) << 23);
  }
}

struct WriteParams {
  KvMap map;
  const uint16_t *kv, *kI, *qI;       // new rows (null: that part is left out)
  uint8_t *kv8, *kI8, *qI8;
  float *kv_scale, *kI_scale, *qI_scale;
  int tokens, T, H_I, d_k, D_I;
  int kv_blocks, kI_blocks;           // blocks of the first two parts; the rest take the queries
  DevErr* err;
};

// Cache row of new token n (position L_b - T + t); -1 for an unmapped page and
// for a sequence shorter than its new tokens (an empty slot of a batch: the
// first rows, or what its stale page table names, may be another's).
template <bool PAGED>
__device__ __forceinline__ long long new_row(const KvMap& map, int n, int T, DevErr* err, bool report) {
  const int b = n / T, t = n - b * T;
  const int pos = map.len(b, report ? err : nullptr, ERR_SITE_CACHE) - T + t;
  if (map.seqlens != nullptr && map.seqlens[b] < T) return -1;   // (reported by len)
  const long long r = map.row<PAGED>(b, pos);
  if (r < 0 && report) report_error(err, DSA_ERR_DEVICE_BOUNDS, ERR_SITE_CACHE | (1u << 8));
  return r;
}

template <int VK, int VI, bool PAGED>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(WriteParams p) {
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  const int gl = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  int blk = blockIdx.x;
  if (blk < p.kv_blocks + p.kI_blocks) {
    const bool keys = blk >= p.kv_blocks;
    if (keys) blk -= p.kv_blocks;
    const int n = blk * kRows + grp;
    const long long r = n < p.tokens ? new_row<PAGED>(p.map, n, p.T, p.err, gl == 0) : -1;
    const int D = keys ? p.D_I : p.d_k;
    const uint16_t* const src[1] = {r >= 0 ? (keys ? p.kI : p.kv) + (size_t)n * D : nullptr};
    uint8_t* const dst[1] = {(keys ? p.kI8 : p.kv8) + r * D};
    float* const sc[1] = {(keys ? p.kI_scale : p.kv_scale) + r};
    if (!keys) quantise_rows<VK, 1>(src, D, dst, sc, gl);
    else quantise_rows<VI, 1>(src, D, dst, sc, gl);
    return;
  }
  blk -= p.kv_blocks + p.kI_blocks;
  const uint16_t* src[kQRows];
  uint8_t* dst[kQRows];
  float* sc[kQRows];
#pragma unroll
  for (int i = 0; i < kQRows; ++i) {
    const long long n = ((long long)blk * kQRows + i) * kRows + grp;
    src[i] = n < (long long)p.tokens * p.H_I ? p.qI + n * p.D_I : nullptr;
    dst[i] = p.qI8 + n * p.D_I;
    sc[i] = p.qI_scale + n;
  }
  quantise_rows<VI, kQRows>(src, p.D_I, dst, sc, gl);
}

struct ReadParams {
  KvMap map;
  const uint8_t *kv8, *kI8;
  const float *kv_scale, *kI_scale;
  uint16_t *kv, *kI;
  int B, begin, count, d_k, D_I;
  int kv_blocks;
  DevErr* err;
};

template <int V>
__device__ __forceinline__ void dequantise_row(const uint8_t* src, float scale, int D, uint16_t* dst, int gl) {
  uint2 v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int col = (j * kLanes + gl) * 8;
    if (col < D) v[j] = *reinterpret_cast<const uint2*>(src + col);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int col = (j * kLanes + gl) * 8;
    if (col >= D) continue;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t two = ((i < 2 ? v[j].x : v[j].y) >> (16 * (i & 1))) & 0xffffu;
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      o[i] = sm100::pack_bf16x2(f.x * scale, f.y * scale);
    }
    *reinterpret_cast<uint4*>(dst + col) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int VK, int VI, bool PAGED>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(ReadParams p) {
  sm100::pdl_launch_dependents();
  sm100::pdl_wait();
  const int gl = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  int blk = blockIdx.x;
  const bool keys = blk >= p.kv_blocks;
  if (keys) blk -= p.kv_blocks;
  const long long n = (long long)blk * kRows + grp;
  if (n >= (long long)p.B * p.count) return;
  const int b = (int)(n / p.count), s = p.begin + (int)(n - (long long)b * p.count);
  if (s >= p.map.len(b, gl == 0 ? p.err : nullptr, ERR_SITE_CACHE)) return;   // past the sequence: left as it is
  const long long r = p.map.row<PAGED>(b, s);
  if (r < 0 && gl == 0) report_error(p.err, DSA_ERR_DEVICE_BOUNDS, ERR_SITE_CACHE | (2u << 8));
  // an unmapped page reads as zeros: row 0's bytes are not touched, the scale is 0 and so are the bytes
  if (r < 0) {
    const int D = keys ? p.D_I : p.d_k;
    uint16_t* dst = (keys ? p.kI : p.kv) + n * D;
    for (int col = gl * 8; col < D; col += kLanes * 8) *reinterpret_cast<uint4*>(dst + col) = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  if (!keys)
    dequantise_row<VK>(p.kv8 + r * p.d_k, p.kv_scale[r], p.d_k, p.kv + n * p.d_k, gl);
  else
    dequantise_row<VI>(p.kI8 + r * p.D_I, p.kI_scale[r], p.D_I, p.kI + n * p.D_I, gl);
}

unsigned blocks_for(long long rows) { return (unsigned)((rows + kRows - 1) / kRows); }

template <int VK, int VI, bool PAGED>
cudaError_t write_t(const LaunchCtx& c, const WriteParams& p, unsigned blocks) {
  const cudaError_t e = launch_pdl(cache_write_kernel<VK, VI, PAGED>, dim3(blocks), dim3(kThreads), 0, c.stream, p);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}
template <int VK, int VI, bool PAGED>
cudaError_t read_t(const LaunchCtx& c, const ReadParams& p, unsigned blocks) {
  const cudaError_t e = launch_pdl(cache_read_kernel<VK, VI, PAGED>, dim3(blocks), dim3(kThreads), 0, c.stream, p);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}

// d_k 576 takes nine vectors of eight columns a lane, 80 two (ten in use);
// D_I 128 two, 64 and 32 one
#define DSA_CACHE8_DISPATCH(fn, c, p, blocks)                                                        \
  (p.map.page_size != 0                                                                              \
       ? (p.d_k > 128 ? (p.D_I > 64 ? fn<9, 2, true>(c, p, blocks) : fn<9, 1, true>(c, p, blocks))   \
                      : (p.D_I > 64 ? fn<2, 2, true>(c, p, blocks) : fn<2, 1, true>(c, p, blocks)))  \
       : (p.d_k > 128 ? (p.D_I > 64 ? fn<9, 2, false>(c, p, blocks) : fn<9, 1, false>(c, p, blocks)) \
                      : (p.D_I > 64 ? fn<2, 2, false>(c, p, blocks) : fn<2, 1, false>(c, p, blocks))))

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// a part is wholly there or wholly absent
bool part_ok(const void* a, const void* b, const void* c) {
  if (a == nullptr && b == nullptr && c == nullptr) return true;
  return a != nullptr && b != nullptr && c != nullptr && aligned16(a) && aligned16(b);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_cache_write(const dsa_shape* s, const uint16_t* kv, uint8_t* kv8, float* kv_scale,
                                      const uint16_t* k_I, uint8_t* kI8, float* kI_scale, const uint16_t* q_I,
                                      uint8_t* qI8, float* qI_scale, void* stream) {
  dsa_status st = api_check_shape(s);
  if (st != DSA_OK) return st;
  if (!part_ok(kv, kv8, kv_scale) || !part_ok(k_I, kI8, kI_scale) || !part_ok(q_I, qI8, qI_scale) ||
      (!kv && !k_I && !q_I))
    return DSA_ERR_INVALID_ARG;
  const long long tokens = (long long)s->B * s->T;
  if (tokens * s->H_I >= (1LL << 31)) return DSA_ERR_UNSUPPORTED;
  LaunchCtx c;
  if ((st = api_make_ctx(stream, &c)) != DSA_OK) return st;
  WriteParams p = {};
  p.map = api_kv_map(s);
  p.kv = kv; p.kv8 = kv8; p.kv_scale = kv_scale;
  p.kI = k_I; p.kI8 = kI8; p.kI_scale = kI_scale;
  p.qI = q_I; p.qI8 = qI8; p.qI_scale = qI_scale;
  p.tokens = (int)tokens; p.T = s->T; p.H_I = s->H_I; p.d_k = s->d_k; p.D_I = s->D_I;
  p.err = c.err;
  p.kv_blocks = kv ? (int)blocks_for(tokens) : 0;
  p.kI_blocks = k_I ? (int)blocks_for(tokens) : 0;
  const unsigned blocks = p.kv_blocks + p.kI_blocks + (q_I ? blocks_for((tokens * s->H_I + kQRows - 1) / kQRows) : 0);
  return DSA_CACHE8_DISPATCH(write_t, c, p, blocks) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

extern "C" dsa_status dsa_cache_read(const dsa_shape* s, int s_begin, int s_count, const uint8_t* kv8,
                                     const float* kv_scale, uint16_t* kv, const uint8_t* kI8, const float* kI_scale,
                                     uint16_t* k_I, void* stream) {
  dsa_status st = api_check_shape(s);
  if (st != DSA_OK) return st;
  if (s_begin < 0 || s_count < 0 || (long long)s_begin + s_count > s->S) return DSA_ERR_INVALID_ARG;
  if (s_count == 0) return DSA_OK;               // empty outputs have no address
  if (!part_ok(kv8, kv, kv_scale) || !part_ok(kI8, k_I, kI_scale) || (!kv && !k_I)) return DSA_ERR_INVALID_ARG;
  if ((long long)s->B * s_count >= (1LL << 31)) return DSA_ERR_UNSUPPORTED;
  LaunchCtx c;
  if ((st = api_make_ctx(stream, &c)) != DSA_OK) return st;
  ReadParams p = {};
  p.map = api_kv_map(s);
  p.kv8 = kv8; p.kv_scale = kv_scale; p.kv = kv;
  p.kI8 = kI8; p.kI_scale = kI_scale; p.kI = k_I;
  p.B = s->B; p.begin = s_begin; p.count = s_count; p.d_k = s->d_k; p.D_I = s->D_I;
  p.err = c.err;
  const long long rows = (long long)s->B * s_count;
  p.kv_blocks = kv ? (int)blocks_for(rows) : 0;
  const unsigned blocks = p.kv_blocks + (k_I ? blocks_for(rows) : 0);
  return DSA_CACHE8_DISPATCH(read_t, c, p, blocks) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
