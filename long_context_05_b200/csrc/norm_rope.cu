// Per-head RMS norm of queries and keys with the rotation by position, in one
// pass over the rows, and its backward pass.
//
// A head row x has D columns.  Its first n are normalised, its last r rotated
// (the two ranges may overlap; then the rotation acts on the normalised row):
//   z_c = w_c x_c rho,  rho = 1 / sqrt(mean_{c < n} x_c^2 + eps)    (c < n; z_c = x_c past n)
//   (y_a, y_b) = (z_a cos - z_b sin, z_a sin + z_b cos),  angle = pos(t) f_i
// over the pairs (a, b) = (i, i + r/2), or (2i, 2i + 1) interleaved, of the
// rotated columns.  Backward, with g = R^T dy the gradient rotated back:
//   dx_c = rho (w_c g_c - x_c rho^2 mean_{c < n}(w g x)),  dw_c = sum over rows of g_c x_c rho.
//
// Nothing is reused between rows but the angles of a token and the weights,
// so the bound is HBM: 4 bytes per element forward, 6 backward.  All rows of
// a side lie one behind the other, so a tile of them is one contiguous piece
// of memory whatever its heads and tokens.  Every warp works by itself: it
// takes a run of tiles of about 4.5 KB and keeps two of them on their way
// into shared memory of its own by bulk copies, so no registers hold loads in
// flight and no warp waits for another.  A row is worked on by G lanes (16 at
// 576 columns, 8 at 128; U rows of each group at a time where rows are short,
// for independent work), reduced by shuffles and written once by 16-byte stores.
// The r/2 sines and cosines of a token are formed once per warp and token.
// The angle is reduced in FP64 (pos times f is exact to 2^-53 there; FP32
// would be off by 2^-24 of the whole angle, half a degree at position 128K),
// then sincospif of the fraction of a turn.
//
// The weight gradients stay in FP32 registers over a warp's rows (a lane
// meets the same columns in every row), are added in a fixed order over the
// block and then over the blocks: the same call gives the same bits.
//
// Measured: 8192 tokens of 129 rows of 576 columns forward 425 us with a cold
// L2, 5.7 TB/s (2.43 GB; 388 us, 6.3 TB/s back to back); 2062 such tokens
// forward and backward 285 us, 5.4 TB/s (265, 5.8); 4096 tokens of 65 rows of
// 128 columns forward and backward 89 us, 3.8 TB/s: short kernels of a dozen
// tiles a warp, where the start and the end weigh.
#include "internal.h"
#include "sm100.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 2;
constexpr int kTileBytes = 4608;    // a warp's tile (both tensors in the backward pass), at most
constexpr int kMaxTileRows = 32;
constexpr int kMaxHalf = 128;       // rotated pairs, at most (r <= 256)
constexpr int kMaxD = 1024;

// kHalf: pairs (i, i + r/2); kInter: pairs (2i, 2i + 1)
enum RopeMode { kNone = 0, kHalf = 1, kInter = 2 };

struct Side {
  const uint16_t* x;     // rows in [tokens, H, D]
  uint16_t* y;           // forward: rows out
  const uint16_t* dy;    // backward: gradient of the rows out
  uint16_t* dx;          // backward: gradient of the rows in
  const float* w;        // [norm_cols] or null (ones)
  float* dw_part;        // backward: [blocks of this side, norm_cols] partial sums
  int H;
  int rows;              // tokens * H
  int tiles;
  int blocks;            // blocks that share the tiles
  float inv_H;
};

struct NrParams {
  Side side[2];
  KvMap map;
  const float* inv_freq;
  int T, D, norm, rope;
  int rt;                // rows of a tile
  int tensor_bytes;      // one tensor's tile in shared memory
  int warp_bytes;        // a warp's stages and angles
  float inv_norm, eps;
  long long wait_ns;
  DevErr* err;
};

// Eight columns as four pairs, for the packed FP32 instructions: half the
// instructions of the scalar ones, and the forward kernel is bound by issue
// as much as by HBM.
struct F8 {
  uint64_t v[4];
};
__device__ __forceinline__ F8 unpack8(const uint4& v) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.v[i] = pair2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  return f;
}
__device__ __forceinline__ uint4 pack8(const F8& f) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpair2(f.v[i]);
    u[i] = pack_bf16x2(x.x, x.y);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
// Weights of the columns 8 i .. 8 i + 7 from their copy in shared memory: the
// first four of every eight, then the second four, so that neighbouring lanes
// read neighbouring 16 bytes.
__device__ __forceinline__ F8 load_w(const ulonglong2* sW, int nvec, int i) {
  const ulonglong2 a = sW[i], b = sW[nvec + i];
  F8 f;
  f.v[0] = a.x; f.v[1] = a.y; f.v[2] = b.x; f.v[3] = b.y;
  return f;
}

// contiguous copy of `bytes` (a multiple of 16) from global to shared memory
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// cos and sin of the angles of tokens [n0, n0 + nt): cs[tt * half + i] (one warp)
__device__ __forceinline__ void fill_angles(const NrParams& p, float2* cs, int n0, int nt) {
  const int half = p.rope >> 1;
  for (int e = threadIdx.x & 31; e < nt * half; e += 32) {
    const int tt = e / half, i = e - tt * half;
    const int n = n0 + tt, b = n / p.T, t = n - b * p.T;
    const int pos = p.map.len(b, i == 0 ? p.err : nullptr, ERR_SITE_NORM) - p.T + t;
    double turns = (double)pos * (double)p.inv_freq[i] * 0.15915494309189535;   // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * (float)turns, &s, &c);
    cs[e] = make_float2(c, s);
  }
}

// Rotate the eight columns rc .. rc + 7 of the rotated range.  kHalf: o holds
// the partner columns rc +- r/2.  back: by the opposite angle.
template <int MODE>
__device__ __forceinline__ void rotate8(F8& z, const F8& o, const float2* cs, int rc, int half, bool back) {
  if constexpr (MODE == kInter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = cs[(rc >> 1) + i], z2 = unpair2(z.v[i]);
      const float s = back ? -a.y : a.y;
      z.v[i] = pair2(z2.x * a.x - z2.y * s, z2.x * s + z2.y * a.x);
    }
  } else if constexpr (MODE == kHalf) {
    const bool first = rc < half;
    const float4* a0 = reinterpret_cast<const float4*>(cs + (first ? rc : rc - half));
    const float sign = first == back ? 1.f : -1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = a0[i];                     // two angles
      z.v[i] = fma2(o.v[i], pair2(a.y * sign, a.w * sign), mul2(z.v[i], pair2(a.x, a.z)));
    }
  }
}

// Blocks of an SM that the registers leave room for.  Long rows want registers
// (140 and 146 at 576 columns; forward 4096 tokens of 129 rows took 235 us
// with five blocks of 96, 229 with four of 128, 196 with three, 261 with two;
// backward 307 with three, 331 and 445 with four and two), short rows warps
// (4096 tokens of 65 rows of 128: 32.9 us with five, 35.5 and 38 with four and
// three; forward and backward 89 with five and four, 96 with five and five;
// forward with pairs (i, i + r/2), which do not fit 96 registers, 40.0 with
// five, 38.6 with four).
constexpr int blocks_per_sm(int V, bool back, bool half) { return V >= 4 ? 3 : back || half ? 4 : 5; }

template <int G, int V, int MODE, bool BACK>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(V, BACK, MODE == kHalf)) norm_rope_kernel(NrParams p) {
  extern __shared__ uint4 smem4[];
  __shared__ uint64_t full_bar[kWarps][kStages];
  constexpr int GP = 32 / G;                      // groups of a warp
  constexpr int U = V <= 2 ? 2 : 1;
  constexpr bool HOIST = V <= 2;                  // weights stay in registers
  constexpr int kTensors = BACK ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % G, grp = lane / G;
  const int sd = (int)blockIdx.x < p.side[0].blocks ? 0 : 1;
  const int blk = blockIdx.x - (sd ? p.side[0].blocks : 0);
  const Side& s = p.side[sd];
  const int half = p.rope >> 1, r0 = p.D - p.rope;
  const unsigned lane_grp = G == 32 ? 0xffffffffu : ((1u << (G & 31)) - 1u) << (grp * G);
  uint8_t* ring = reinterpret_cast<uint8_t*>(smem4) + warp * p.warp_bytes;
  float2* cs = reinterpret_cast<float2*>(ring + kStages * kTensors * p.tensor_bytes);
  uint64_t* full = full_bar[warp];
  const int workers = s.blocks * kWarps, me = blk * kWarps + warp;
  const int tile0 = (int)((long long)s.tiles * me / workers), tile1 = (int)((long long)s.tiles * (me + 1) / workers);
  const bool need_x = !BACK || p.norm > 0;
  auto load_tile = [&](int tile) {
    const int st = (tile - tile0) % kStages;
    const uint32_t bytes = (uint32_t)min(p.rt, s.rows - tile * p.rt) * p.D * 2;
    const size_t at = (size_t)tile * p.rt * p.D;
    mbar_arrive_expect_tx(&full[st], bytes * (BACK && need_x ? 2 : 1));
    uint8_t* d = ring + st * kTensors * p.tensor_bytes;
    bulk_load(d, (BACK ? s.dy : s.x) + at, bytes, &full[st]);
    if (BACK && need_x) bulk_load(d + p.tensor_bytes, s.x + at, bytes, &full[st]);
  };
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  // What follows on the stream may start: at once where rows are short (a
  // training pass of 4096 tokens of 65 rows of 128: 89.6 us, 91.3 at the end),
  // behind the tiles where they are long (2062 tokens of 129 rows of 576: 265
  // us, 269 at the start).
  if (V < 4) pdl_launch_dependents();
  pdl_wait();                                     // nothing of global memory is read before this
  if (lane == 0) {
    for (int i = tile0; i < tile1 && i < tile0 + kStages; ++i) load_tile(i);
  }
  __syncwarp();
  // the weights' copy, behind the warps' rings (ones where there are none)
  const int nvec = p.norm >> 3;
  ulonglong2* sW = reinterpret_cast<ulonglong2*>(reinterpret_cast<uint8_t*>(smem4) + kWarps * p.warp_bytes);
  for (int i = threadIdx.x; i < 2 * nvec; i += kThreads) {
    const float4 w4 = s.w != nullptr ? __ldg(reinterpret_cast<const float4*>(s.w) + i) : make_float4(1.f, 1.f, 1.f, 1.f);
    *reinterpret_cast<float4*>(sW + (i & 1) * nvec + (i >> 1)) = w4;
  }
  __syncthreads();
  F8 wr[HOIST ? V : 1];
  if constexpr (HOIST) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if ((j * G + gl) * 8 < p.norm) wr[j] = load_w(sW, nvec, j * G + gl);
  }
  auto weights = [&](int j) -> F8 {
    if constexpr (HOIST) return wr[j];
    else return load_w(sW, nvec, j * G + gl);
  };
  // steps of G * 8 columns that lie wholly in the normalised columns, and of
  // those the ones with no rotated column: there no lane decides for itself
  const int jn = p.norm / (G * 8), jf = min(p.norm, MODE == kNone ? p.D : r0) / (G * 8);
  F8 acc[BACK ? V : 1];
  if constexpr (BACK) {
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j].v[i] = 0ull;
  }
  const AbortSources no_abort{nullptr, nullptr};
  int n_lo = 0, n_cnt = 0;                        // tokens whose angles cs holds
  // the tile's first row is head `off` of token n0; small numbers are divided
  // by H through its reciprocal (both below 2^11: exact, with the half)
  auto by_H = [&](int x) { return (int)(((float)x + 0.5f) * s.inv_H); };
  int n0 = tile0 * p.rt / s.H, off = tile0 * p.rt - n0 * s.H;
  bool ok = true;
  for (int tile = tile0; tile < tile1; ++tile) {
    const int st = (tile - tile0) % kStages;
    const int row0 = tile * p.rt, nr = min(p.rt, s.rows - row0);
    if (MODE != kNone) {
      const int nt = by_H(off + nr - 1) + 1;
      if (n0 < n_lo || n0 + nt > n_lo + n_cnt) {
        fill_angles(p, cs, n0, nt);
        n_lo = n0;
        n_cnt = nt;
        __syncwarp();
      }
    }
    ok = __all_sync(0xffffffffu, mbar_wait(&full[st], (uint32_t)((tile - tile0) / kStages) & 1, p.wait_ns, no_abort));
    if (!ok) {
      if (lane == 0) report_error(p.err, DSA_ERR_TIMEOUT, ERR_SITE_NORM | (2u << 8));
      // the copies still on their way, with the same limit
      for (int i = tile + 1; i < tile1 && i < tile + kStages; ++i)
        mbar_wait(&full[(i - tile0) % kStages], (uint32_t)((i - tile0) / kStages) & 1, p.wait_ns, no_abort);
      break;
    }
    const uint8_t* sA = ring + st * kTensors * p.tensor_bytes;     // x forward, dy backward
    for (int rr = 0; rr < nr; rr += GP * U) {
      int r[U];
      const uint4* ra[U];                          // this lane's first columns of the row
      uint64_t ss2[U], dot2[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        r[u] = min(rr + u * GP + grp, nr - 1);    // groups past the tile follow its last row and write nothing
        ra[u] = reinterpret_cast<const uint4*>(sA + r[u] * p.D * 2) + gl;
        ss2[u] = dot2[u] = 0ull;
      }
      // the angles of row r: its token within those of cs
      auto angles = [&](int r_) -> const float2* { return cs + (n0 - n_lo + by_H(off + r_)) * half; };
      // columns `col` of the partner range (col rotated)
      auto partner = [&](int u, int col) -> F8 {
        const int pc = col - r0 < half ? col + half : col - half;
        return unpack8(ra[u][(pc >> 3) - gl]);
      };
      // backward: g = R^T dy at this lane's columns of step j
      auto rotated = [&](int u, int j, int col) -> F8 {
        F8 f = unpack8(ra[u][j * G]);
        if (MODE != kNone && col >= r0) {
          F8 q = f;
          if constexpr (MODE == kHalf) q = partner(u, col);
          rotate8<MODE>(f, q, angles(r[u]), col - r0, half, true);
        }
        return f;
      };
      auto x_of = [&](int u, int j) -> F8 {
        return unpack8(*reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(ra[u] + j * G) + p.tensor_bytes));
      };
      // 1. the sums of squares, backward also of w g x
      F8 x[BACK ? 1 : U][BACK ? 1 : V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * G + gl) * 8;
        if constexpr (!BACK) {
          if (j < jn || col < p.D) {
#pragma unroll
            for (int u = 0; u < U; ++u) x[u][j] = unpack8(ra[u][j * G]);
          }
          if (j < jn || col < p.norm) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) ss2[u] = fma2(x[u][j].v[i], x[u][j].v[i], ss2[u]);
          }
        } else if (j < jn || col < p.norm) {
          const F8 w = weights(j);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const F8 f = j < jf ? unpack8(ra[u][j * G]) : rotated(u, j, col), xr = x_of(u, j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              ss2[u] = fma2(xr.v[i], xr.v[i], ss2[u]);
              dot2[u] = fma2(mul2(f.v[i], xr.v[i]), w.v[i], dot2[u]);
            }
          }
        }
      }
      float ss[U], dot[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float2 a = unpair2(ss2[u]), d = unpair2(dot2[u]);
        ss[u] = a.x + a.y;
        dot[u] = d.x + d.y;
      }
#pragma unroll
      for (int d = 1; d < G; d <<= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          ss[u] += __shfl_xor_sync(lane_grp, ss[u], d);
          if (BACK) dot[u] += __shfl_xor_sync(lane_grp, dot[u], d);
        }
      uint64_t rho[U], c1[U];
      uint4* dst[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float h = rsqrtf(fmaf(ss[u], p.inv_norm, p.eps));
        // (in this order no step passes FP32: h^3 alone does for rows of 1e-13)
        const float c = -(dot[u] * p.inv_norm * h * h * h);
        rho[u] = pair2(h, h);
        c1[u] = pair2(c, c);
        dst[u] = reinterpret_cast<uint4*>((BACK ? s.dx : s.y) + (size_t)(row0 + r[u]) * p.D) + gl;
      }
      // dx at normalised columns, from g and x; the weight sums
      auto grad = [&](int u, int j, const F8& f, const F8& w) -> F8 {
        const F8 xr = x_of(u, j);
        F8 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t gr = mul2(f.v[i], rho[u]);
          acc[BACK ? j : 0].v[i] = fma2(gr, xr.v[i], acc[BACK ? j : 0].v[i]);
          o.v[i] = fma2(gr, w.v[i], mul2(c1[u], xr.v[i]));
        }
        return o;
      };
      const bool whole = rr + GP * U <= nr;        // the same for the warp
      auto live = [&](int u) { return whole || rr + u * GP + grp < nr; };
      // 2. the rows out
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * G + gl) * 8;
        if (j < jf) {
          const F8 w = weights(j);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (!live(u)) continue;
            F8 o;
            if constexpr (BACK) {
              o = grad(u, j, unpack8(ra[u][j * G]), w);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) o.v[i] = mul2(mul2(x[u][j].v[i], rho[u]), w.v[i]);
            }
            dst[u][j * G] = pack8(o);
          }
        } else if (col < p.D) {
          const bool rot = MODE != kNone && col >= r0, nrm = col < p.norm;
          F8 w = {};
          if (nrm) w = weights(j);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (!live(u)) continue;
            F8 f;
            if constexpr (BACK) {
              f = rotated(u, j, col);
              if (nrm) f = grad(u, j, f, w);
            } else {
              f = x[u][j];
              if (nrm) {
#pragma unroll
                for (int i = 0; i < 4; ++i) f.v[i] = mul2(mul2(f.v[i], rho[u]), w.v[i]);
              }
              if (rot) {
                F8 g = f;
                if constexpr (MODE == kHalf) {
                  const int pc = col - r0 < half ? col + half : col - half;
                  g = partner(u, col);
                  if (pc < p.norm) {
                    const F8 wp = load_w(sW, nvec, pc >> 3);
#pragma unroll
                    for (int i = 0; i < 4; ++i) g.v[i] = mul2(mul2(g.v[i], rho[u]), wp.v[i]);
                  }
                }
                rotate8<MODE>(f, g, angles(r[u]), col - r0, half, false);
              }
            }
            dst[u][j * G] = pack8(f);
          }
        }
      }
    }
    __syncwarp();                                 // the stage is read
    if (lane == 0 && tile + kStages < tile1) load_tile(tile + kStages);
    const int q = by_H(off + p.rt);
    n0 += q;
    off += p.rt - q * s.H;
  }
  if (V >= 4) pdl_launch_dependents();
  if constexpr (BACK) {
    if (s.dw_part == nullptr) return;
    // the groups' sums, in group order: first over the groups of a warp by
    // shuffles, then over the warps through shared memory (every tile has landed)
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem4);  // [kWarps][G * V * 8]
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 two = unpair2(acc[j].v[i / 2]);
        float a = i & 1 ? two.y : two.x;
#pragma unroll
        for (int d = G; d < 32; d <<= 1) a += __shfl_xor_sync(0xffffffffu, a, d);
        if (lane < G) red[warp * (G * V * 8) + (j * G + gl) * 8 + i] = a;
      }
    __syncthreads();
    for (int c = threadIdx.x; c < p.norm; c += kThreads) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) a += red[w * (G * V * 8) + c];
      s.dw_part[(size_t)blk * p.norm + c] = a;
    }
  }
}

// dw[c] = sum over a side's blocks, in block order: 8 columns per block of 256
// threads, 32 lanes over the partial rows
struct DwParams {
  const float* part[2];
  float* dw[2];
  int blocks[2];
  int norm;
};
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(DwParams p) {
  __shared__ float red[32][9];
  const int sd = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  if (p.dw[sd] == nullptr) return;
  const int c = blockIdx.x * 8 + (threadIdx.x & 7), l = threadIdx.x >> 3;
  float a = 0.f;
  if (c < p.norm)
    for (int i = l; i < p.blocks[sd]; i += 32) a += p.part[sd][(size_t)i * p.norm + c];
  red[l][threadIdx.x & 7] = a;
  __syncthreads();
  if (threadIdx.x < 8 && c < p.norm) {
    float t = 0.f;
    for (int i = 0; i < 32; ++i) t += red[i][threadIdx.x];
    p.dw[sd][c] = t;
  }
}

// Lanes of a row: few, so that a warp's shuffles, square roots and addresses
// serve many rows, with at most five steps of registers each.
int lanes_of(int D) { return D <= 64 ? 4 : D <= 128 ? 8 : D <= 640 ? 16 : 32; }

int rows_at_once(int D) { return 32 / lanes_of(D) * (D <= 256 ? 2 : 1); }   // GP * U of the kernel

// Rows of a tile: kTileBytes of them (half that for short rows, which need
// more warps and less each: 99 -> 94 us on 4096 tokens of 65 heads of 128),
// in full steps of a warp.
int tile_rows(int D, bool back) {
  const int g = rows_at_once(D);
  int rt = (D <= 256 ? kTileBytes / 2 : kTileBytes) / (D * (back ? 4 : 2)) / g * g;
  if (rt > kMaxTileRows) rt = kMaxTileRows;
  return rt < g ? g : rt;
}

// Tokens that a tile of a side with H heads touches, at most.
int tile_tokens(int rt, int H) { return H == 0 ? 0 : H == 1 ? rt : (rt - 2) / H + 2; }

int tensor_bytes_of(int D, bool back) { return (tile_rows(D, back) * D * 2 + 127) / 128 * 128; }

int warp_bytes_of(const dsa_norm_rope_desc* d, bool back) {
  const int rt = tile_rows(d->D, back);
  const int tq = tile_tokens(rt, d->Hq), tk = tile_tokens(rt, d->Hk);
  const int angles = (tq > tk ? tq : tk) * (d->rope_cols / 2) * (int)sizeof(float2);
  return kStages * (back ? 2 : 1) * tensor_bytes_of(d->D, back) + (angles + 127) / 128 * 128;
}

size_t smem_of(const dsa_norm_rope_desc* d, bool back) {
  const size_t n = (size_t)kWarps * warp_bytes_of(d, back) + (size_t)d->norm_cols * sizeof(float);
  const size_t red = back ? (size_t)kWarps * 1024 * sizeof(float) : 0;   // at most: G V 8 <= 1024
  return n > red ? n : red;
}

// Blocks resident at once: what shared memory and registers allow.
int resident_blocks(const dsa_norm_rope_desc* d, bool back, int num_sms) {
  int n = (int)(227 * 1024 / (smem_of(d, back) + 1280));
  const int regs = blocks_per_sm(d->D > 256 ? 4 : 1, back, d->rope_cols > 0 && d->interleaved == 0);
  if (n > regs) n = regs;
  return (n < 1 ? 1 : n) * num_sms;
}

// The resident blocks shared between the sides by rows (a token's angles count
// as one more), each side that has rows with at least one and no more than
// one tile a warp makes use of.
void plan(NrParams* p, int tokens, int resident) {
  const long long all = p->side[0].H + p->side[1].H + 2;
  for (Side& s : p->side) {
    s.rows = tokens * s.H;
    s.tiles = (s.rows + p->rt - 1) / p->rt;
    s.inv_H = s.H > 0 ? 1.f / (float)s.H : 0.f;
    long long n = s.H == 0 ? 0 : (long long)resident * (s.H + 1) / all;
    if (s.H > 0 && n < 1) n = 1;
    const int most = (s.tiles + kWarps - 1) / kWarps;
    s.blocks = (int)(n < most ? n : most);
  }
}

template <int G, int V, int MODE, bool BACK>
cudaError_t launch_mode(const LaunchCtx& c, const NrParams& p, size_t smem) {
  auto kern = norm_rope_kernel<G, V, MODE, BACK>;
  static std::atomic<int> granted[kMaxDevices];
  // Kernels of three blocks an SM ask for all of its shared memory: one that
  // starts beside the end of the other, where that one has divided the memory
  // for its own needs, had room for two (a forward and a backward pass in turn
  // took 330 us, 101 and 160 alone).  Those of short rows fill it anyway, and
  // took 92 us instead of 90 with it.
  const cudaError_t e = grant_smem(kern, (int)smem, c.device, granted, V >= 4);
  if (e != cudaSuccess) return e;
  const cudaError_t l = launch_pdl(kern, dim3((unsigned)(p.side[0].blocks + p.side[1].blocks)), dim3(kThreads), smem,
                                   c.stream, p);
  if (l != cudaSuccess) return l;
  note_launches(1);
  return cudaGetLastError();
}
template <int G, int V>
cudaError_t launch_gv(const LaunchCtx& c, const NrParams& p, bool inter, bool back, size_t sm) {
  if (p.rope == 0) return back ? launch_mode<G, V, kNone, true>(c, p, sm) : launch_mode<G, V, kNone, false>(c, p, sm);
  if (inter) return back ? launch_mode<G, V, kInter, true>(c, p, sm) : launch_mode<G, V, kInter, false>(c, p, sm);
  return back ? launch_mode<G, V, kHalf, true>(c, p, sm) : launch_mode<G, V, kHalf, false>(c, p, sm);
}
cudaError_t launch_nr(const LaunchCtx& c, const NrParams& p, const dsa_norm_rope_desc* d, bool back) {
  const bool inter = d->interleaved != 0;
  const size_t sm = smem_of(d, back);
  if (p.D <= 64) return launch_gv<4, 2>(c, p, inter, back, sm);
  if (p.D <= 128) return launch_gv<8, 2>(c, p, inter, back, sm);
  if (p.D <= 256) return launch_gv<16, 2>(c, p, inter, back, sm);
  if (p.D <= 640) return launch_gv<16, 5>(c, p, inter, back, sm);
  return launch_gv<32, 4>(c, p, inter, back, sm);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

dsa_status check_desc(const dsa_shape* s, const dsa_norm_rope_desc* d) {
  dsa_status st = api_check_shape(s);
  if (st != DSA_OK) return st;
  if (d == nullptr || d->Hq < 0 || d->Hk < 0 || d->D <= 0 || d->norm_cols < 0 || d->rope_cols < 0)
    return DSA_ERR_INVALID_ARG;
  if (d->Hq + d->Hk == 0 || d->norm_cols > d->D || d->rope_cols > d->D) return DSA_ERR_INVALID_ARG;
  if (d->rope_cols > 0 && d->inv_freq == nullptr) return DSA_ERR_INVALID_ARG;
  if (d->norm_cols > 0 && !(d->eps >= 0.f)) return DSA_ERR_INVALID_ARG;
  if ((d->q_weight && !aligned16(d->q_weight)) || (d->k_weight && !aligned16(d->k_weight))) return DSA_ERR_INVALID_ARG;
  if (d->D % 8 != 0 || d->D > kMaxD || d->norm_cols % 8 != 0 || d->rope_cols % 16 != 0 ||
      d->rope_cols > 2 * kMaxHalf || d->Hq > 1024 || d->Hk > 1024)
    return DSA_ERR_UNSUPPORTED;
  // rows of a launch count as an int
  if ((long long)s->B * s->T * (d->Hq + d->Hk) >= (1LL << 31) - kMaxTileRows) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

NrParams make_params(const LaunchCtx& c, const dsa_shape* s, const dsa_norm_rope_desc* d, bool back) {
  NrParams p = {};
  p.map = api_kv_map(s);
  p.inv_freq = d->inv_freq;
  p.T = s->T;
  p.D = d->D;
  p.norm = d->norm_cols;
  p.rope = d->rope_cols;
  p.rt = tile_rows(d->D, back);
  p.tensor_bytes = tensor_bytes_of(d->D, back);
  p.warp_bytes = warp_bytes_of(d, back);
  p.inv_norm = d->norm_cols > 0 ? 1.f / (float)d->norm_cols : 0.f;
  p.eps = d->eps;
  p.wait_ns = c.wait_ns;
  p.err = c.err;
  p.side[0].H = d->Hq;
  p.side[1].H = d->Hk;
  p.side[0].w = d->q_weight;
  p.side[1].w = d->k_weight;
  plan(&p, s->B * s->T, resident_blocks(d, back, c.num_sms));
  return p;
}

bool rows_ok(int H, const void* a, const void* b) {
  return H == 0 || (a != nullptr && b != nullptr && aligned16(a) && aligned16(b));
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" size_t dsa_norm_rope_workspace_size(const dsa_shape* s, const dsa_norm_rope_desc* d) {
  if (check_desc(s, d) != DSA_OK) return 0;
  // a row of partial sums for each resident block, one more for a side that
  // would have had none; sized for 256 SMs, so that it depends on no device
  return ((size_t)resident_blocks(d, true, 256) + 2) * (d->norm_cols > 0 ? d->norm_cols : 1) * sizeof(float);
}

extern "C" dsa_status dsa_norm_rope(const dsa_shape* s, const dsa_norm_rope_desc* d, const uint16_t* q,
                                    const uint16_t* k, uint16_t* q_out, uint16_t* k_out, void* stream) {
  dsa_status st = check_desc(s, d);
  if (st != DSA_OK) return st;
  if (!rows_ok(d->Hq, q, q_out) || !rows_ok(d->Hk, k, k_out)) return DSA_ERR_INVALID_ARG;
  LaunchCtx c;
  if ((st = api_make_ctx(stream, &c)) != DSA_OK) return st;
  NrParams p = make_params(c, s, d, false);
  p.side[0].x = q;
  p.side[0].y = q_out;
  p.side[1].x = k;
  p.side[1].y = k_out;
  return launch_nr(c, p, d, false) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

extern "C" dsa_status dsa_norm_rope_backward(const dsa_shape* s, const dsa_norm_rope_desc* d, const uint16_t* q,
                                             const uint16_t* k, const uint16_t* dq_out, const uint16_t* dk_out,
                                             uint16_t* dq, uint16_t* dk, float* dq_weight, float* dk_weight, void* ws,
                                             size_t ws_bytes, void* stream) {
  dsa_status st = check_desc(s, d);
  if (st != DSA_OK) return st;
  if (!rows_ok(d->Hq, dq_out, dq) || !rows_ok(d->Hk, dk_out, dk)) return DSA_ERR_INVALID_ARG;
  if (d->norm_cols > 0 && (!rows_ok(d->Hq, q, q) || !rows_ok(d->Hk, k, k))) return DSA_ERR_INVALID_ARG;
  LaunchCtx c;
  if ((st = api_make_ctx(stream, &c)) != DSA_OK) return st;
  if (c.num_sms > 256) return DSA_ERR_UNSUPPORTED;
  NrParams p = make_params(c, s, d, true);
  p.side[0].x = q;
  p.side[0].dy = dq_out;
  p.side[0].dx = dq;
  p.side[1].x = k;
  p.side[1].dy = dk_out;
  p.side[1].dx = dk;
  DwParams w = {};
  w.norm = p.norm;
  if (p.norm > 0 && (dq_weight != nullptr || dk_weight != nullptr)) {
    if (ws == nullptr || ws_bytes < dsa_norm_rope_workspace_size(s, d) || (reinterpret_cast<uintptr_t>(ws) & 3u))
      return DSA_ERR_WORKSPACE;
    float* part = static_cast<float*>(ws);
    float* dw[2] = {dq_weight, dk_weight};         // a side without heads: the sum over no rows
    for (int i = 0; i < 2; ++i) {
      if (dw[i] == nullptr) continue;
      p.side[i].dw_part = part;
      w.part[i] = part;
      w.dw[i] = dw[i];
      w.blocks[i] = p.side[i].blocks;
      part += (size_t)p.side[i].blocks * p.norm;
    }
  }
  if (launch_nr(c, p, d, true) != cudaSuccess) return DSA_ERR_CUDA;
  if (w.dw[0] != nullptr || w.dw[1] != nullptr) {
    if (launch_pdl(norm_rope_dw_kernel, dim3((unsigned)((p.norm + 7) / 8), 2), dim3(256), 0, c.stream, w) != cudaSuccess)
      return DSA_ERR_CUDA;
    note_launches(1);
    if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  }
  return DSA_OK;
}
