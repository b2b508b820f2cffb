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
// so the bound is HBM: 4 bytes per element forward, 6 backward.  A row is
// held in the registers of G lanes (16 up to 640 columns: a 16-byte load of
// each covers 256 contiguous bytes of a row), read once, reduced by shuffles
// and written once.  The pair of a rotated column comes from another lane by
// shuffles where it lies in the same step of 16 G bytes, else it is read again
// (from L1).  The r/2 sines and cosines of a token are
// formed once per block, in shared memory, for all heads the block handles.
// The angle is reduced in FP64 (pos times f is exact to 2^-53 there; FP32
// would be off by 2^-24 of the whole angle, half a degree at position 128K),
// then sincospif of the fraction of a turn.
//
// The weight gradients stay in FP32 registers over a block's rows (a lane
// meets the same columns in every row), are added in a fixed order over the
// block and then over the blocks: the same call gives the same bits.
#include "internal.h"
#include "sm100.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 128;
constexpr int kTileTokens = 16;   // tokens whose angles a block holds at a time, at most
constexpr int kMaxHalf = 128;     // rotated pairs, at most (r <= 256)
constexpr int kMaxD = 1024;

// kHalf: pairs (i, i + r/2), the partner read again; kShfl: the same with the
// partner columns in lane ^ (r / 16) of the same step; kInter: pairs (2i, 2i + 1)
enum RopeMode { kNone = 0, kHalf = 1, kInter = 2, kShfl = 3 };

struct Side {
  const uint16_t* x;     // rows in [tokens, H, D]
  uint16_t* y;           // forward: rows out
  const uint16_t* dy;    // backward: gradient of the rows out
  uint16_t* dx;          // backward: gradient of the rows in
  const float* w;        // [norm_cols] or null (ones)
  float* dw_part;        // backward: [blocks of this side, norm_cols] partial sums
  int H;
  int tile;              // tokens of an item
  int hc;                // heads of an item
  int items;             // work items of this side
  int hsplit;            // items per token tile
  int blocks;            // backward: blocks of this side
};

struct NrParams {
  Side side[2];
  KvMap map;
  const float* inv_freq;
  int tokens, T, D, norm, rope;
  float inv_norm, eps;
  DevErr* err;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(sm100::pack_bf16x2(f[0], f[1]), sm100::pack_bf16x2(f[2], f[3]), sm100::pack_bf16x2(f[4], f[5]),
                    sm100::pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void load_w(const float* w, int col, float (&f)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
    return;
  }
  const float4 a = __ldg(reinterpret_cast<const float4*>(w + col)), b = __ldg(reinterpret_cast<const float4*>(w + col) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// cos and sin of the angles of tokens [n0, n0 + nt): cs[tt * half + i]
__device__ __forceinline__ void fill_angles(const NrParams& p, float2* cs, int n0, int nt) {
  const int half = p.rope >> 1;
  for (int e = threadIdx.x; e < nt * half; e += kThreads) {
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

// Rotate the eight columns at `col` (offset rc = col - (D - r) >= 0 into the
// rotated range).  kHalf, kShfl: o holds the partner columns rc +- r/2.  back: by
// the opposite angle.
template <int MODE>
__device__ __forceinline__ void rotate8(float (&z)[8], const float (&o)[8], const float2* cs, int rc, int half,
                                        bool back) {
  if constexpr (MODE == kInter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = cs[(rc >> 1) + i];
      const float s = back ? -a.y : a.y;
      const float u = z[2 * i], v = z[2 * i + 1];
      z[2 * i] = u * a.x - v * s;
      z[2 * i + 1] = u * s + v * a.x;
    }
  } else if constexpr (MODE == kHalf || MODE == kShfl) {
    const bool first = rc < half;
    const float2* a0 = cs + (first ? rc : rc - half);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 a = a0[i];
      float s = back ? -a.y : a.y;
      if (first) s = -s;
      z[i] = fmaf(o[i], s, z[i] * a.x);
    }
  }
}

// which side and item this block works on: the q side's items come first
__device__ __forceinline__ void item_of(const Side& s, int tokens, int item, int& n0, int& nt, int& h0, int& hn) {
  const int tile = item / s.hsplit, hs = item - tile * s.hsplit;
  n0 = tile * s.tile;
  nt = min(s.tile, tokens - n0);
  h0 = hs * s.hc;
  hn = min(s.hc, s.H - h0);
}

template <int G, int V, int MODE>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(NrParams p) {
  extern __shared__ float2 cs[];
  constexpr int kRows = kThreads / G;             // rows in flight in the block
  const int gl = threadIdx.x % G, grp = threadIdx.x / G;
  int item = blockIdx.x;
  const int sd = item < p.side[0].items ? 0 : 1;
  if (sd) item -= p.side[0].items;
  const Side& s = p.side[sd];
  int n0, nt, h0, hn;
  item_of(s, p.tokens, item, n0, nt, h0, hn);
  if (MODE != kNone) {
    fill_angles(p, cs, n0, nt);
    __syncthreads();
  }
  const int half = p.rope >> 1, r0 = p.D - p.rope;
  const int nrows = nt * hn;
  const unsigned lane_grp = G == 32 ? 0xffffffffu : ((1u << (G & 31)) - 1u) << ((threadIdx.x & 31) / G * G);
  for (int rr = 0; rr < nrows; rr += kRows) {
    const bool on = rr + grp < nrows;
    const int r = on ? rr + grp : rr;             // idle groups read and write nothing
    const int tt = r / hn, h = h0 + r - tt * hn;
    const size_t base = ((size_t)(n0 + tt) * s.H + h) * p.D;
    const uint16_t* x = s.x + base;
    uint4 v[V], o[MODE == kHalf ? V : 1];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * G + gl) * 8;
      v[j] = make_uint4(0u, 0u, 0u, 0u);
      if (on && col < p.D) v[j] = *reinterpret_cast<const uint4*>(x + col);
      if constexpr (MODE == kHalf) {
        // the partner columns, read (from L1) before any lane writes the row
        if (on && col < p.D && col >= r0) o[j] = *reinterpret_cast<const uint4*>(x + (col - r0 < half ? col + half : col - half));
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if ((j * G + gl) * 8 < p.norm) {
        float f[8];
        unpack8(v[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
      }
    }
#pragma unroll
    for (int d = 1; d < G; d <<= 1) ss += __shfl_xor_sync(lane_grp, ss, d);
    __syncwarp(lane_grp);                         // every lane holds its columns: the row may be written over
    const float rho = rsqrtf(fmaf(ss, p.inv_norm, p.eps));
    uint16_t* y = s.y + base;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * G + gl) * 8;
      float f[8], g[8];
      unpack8(v[j], f);
      if (col < p.norm) {
        float w[8];
        load_w(s.w, col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= rho * w[i];
      }
      if constexpr (MODE == kShfl) {
        // every lane of the row takes part in a step that holds rotated columns
        if ((j * G + G) * 8 > r0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = __shfl_xor_sync(lane_grp, f[i], half >> 3);
        }
      }
      if (!on || col >= p.D) continue;
      if (MODE != kNone && col >= r0) {
        if constexpr (MODE == kHalf) {
          const int pc = col - r0 < half ? col + half : col - half;
          unpack8(o[j], g);
          if (pc < p.norm) {
            float w[8];
            load_w(s.w, pc, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] *= rho * w[i];
          }
        }
        rotate8<MODE>(f, g, cs + tt * half, col - r0, half, false);
      } else if (p.norm <= col) {
        *reinterpret_cast<uint4*>(y + col) = v[j];
        continue;
      }
      *reinterpret_cast<uint4*>(y + col) = pack8(f);
    }
  }
}

// Backward.  A block keeps to one side and takes its items in turn; the grid
// is what is resident at once, so that every block has an equal share.
template <int V>
constexpr int bwd_blocks_per_sm() { return V >= 4 ? 3 : 6; }
template <int G, int V, int MODE>
__global__ void __launch_bounds__(kThreads, bwd_blocks_per_sm<V>()) norm_rope_bwd_kernel(NrParams p) {
  extern __shared__ float2 cs[];
  constexpr int kRows = kThreads / G;
  const int gl = threadIdx.x % G, grp = threadIdx.x / G;
  const int sd = (int)blockIdx.x < p.side[0].blocks ? 0 : 1;
  const int blk = blockIdx.x - (sd ? p.side[0].blocks : 0);
  const Side& s = p.side[sd];
  const int half = p.rope >> 1, r0 = p.D - p.rope;
  const unsigned lane_grp = G == 32 ? 0xffffffffu : ((1u << (G & 31)) - 1u) << ((threadIdx.x & 31) / G * G);
  float acc[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.f;
  for (int item = blk; item < s.items; item += s.blocks) {
    int n0, nt, h0, hn;
    item_of(s, p.tokens, item, n0, nt, h0, hn);
    if (MODE != kNone) {
      __syncthreads();                            // the last item's angles are no longer read
      fill_angles(p, cs, n0, nt);
      __syncthreads();
    }
    const int nrows = nt * hn;
    for (int rr = 0; rr < nrows; rr += kRows) {
      const bool on = rr + grp < nrows;
      const int r = on ? rr + grp : rr;
      const int tt = r / hn, h = h0 + r - tt * hn;
      const size_t base = ((size_t)(n0 + tt) * s.H + h) * p.D;
      uint4 v[V], g[V], o[MODE == kHalf ? V : 1];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * G + gl) * 8;
        v[j] = make_uint4(0u, 0u, 0u, 0u);
        g[j] = make_uint4(0u, 0u, 0u, 0u);
        if (on && col < p.D) {
          g[j] = *reinterpret_cast<const uint4*>(s.dy + base + col);
          if (col < p.norm) v[j] = *reinterpret_cast<const uint4*>(s.x + base + col);
          if constexpr (MODE == kHalf) {
            if (col >= r0)
              o[j] = *reinterpret_cast<const uint4*>(s.dy + base + (col - r0 < half ? col + half : col - half));
          }
        }
      }
      // g = R^T dy, kept in FP32 where it was rotated and also normalised;
      // ss = sum x^2, dot = sum w g x
      float ss = 0.f, dot = 0.f;
      auto rotated = [&](int j, int col, float (&f)[8]) {
        unpack8(g[j], f);
        float q[8];
        if constexpr (MODE == kHalf) unpack8(o[j], q);
        if constexpr (MODE == kShfl) {
          if ((j * G + G) * 8 > r0) {
            uint4 x;
            x.x = __shfl_xor_sync(lane_grp, g[j].x, half >> 3);
            x.y = __shfl_xor_sync(lane_grp, g[j].y, half >> 3);
            x.z = __shfl_xor_sync(lane_grp, g[j].z, half >> 3);
            x.w = __shfl_xor_sync(lane_grp, g[j].w, half >> 3);
            unpack8(x, q);
          }
        }
        if (MODE != kNone && col >= r0 && col < p.D) rotate8<MODE>(f, q, cs + tt * half, col - r0, half, true);
      };
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * G + gl) * 8;
        if (j * G * 8 < p.norm) {                // the same for every lane of the row
          float f[8], xf[8], w[8];
          rotated(j, col, f);
          if (col >= p.norm) continue;
          unpack8(v[j], xf);
          load_w(s.w, col, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(xf[i], xf[i], ss);
            dot = fmaf(f[i] * xf[i], w[i], dot);
          }
        }
      }
#pragma unroll
      for (int d = 1; d < G; d <<= 1) {
        ss += __shfl_xor_sync(lane_grp, ss, d);
        dot += __shfl_xor_sync(lane_grp, dot, d);
      }
      __syncwarp(lane_grp);                       // every lane holds its columns: dx may be dy's buffer
      const float rho = rsqrtf(fmaf(ss, p.inv_norm, p.eps));
      const float c1 = rho * rho * rho * dot * p.inv_norm;
      uint16_t* dx = s.dx + base;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * G + gl) * 8;
        float f[8];
        rotated(j, col, f);
        if (!on || col >= p.D) continue;
        if (col < p.norm) {
          float xf[8], w[8];
          unpack8(v[j], xf);
          load_w(s.w, col, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[j][i] = fmaf(f[i] * rho, xf[i], acc[j][i]);
            f[i] = fmaf(rho * w[i], f[i], -c1 * xf[i]);
          }
        }
        *reinterpret_cast<uint4*>(dx + col) = pack8(f);
      }
    }
  }
  if (s.dw_part == nullptr) return;
  // the groups' sums, in group order: first over the groups of a warp by
  // shuffles, then over the warps through shared memory
  __syncthreads();
  float* red = reinterpret_cast<float*>(cs);      // [kThreads / 32][G * V * 8]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a = acc[j][i];
#pragma unroll
      for (int d = G; d < 32; d <<= 1) a += __shfl_xor_sync(0xffffffffu, a, d);
      if (lane < G) red[warp * (G * V * 8) + (j * G + gl) * 8 + i] = a;
    }
  __syncthreads();
  for (int c = threadIdx.x; c < p.norm; c += kThreads) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) a += red[w * (G * V * 8) + c];
    s.dw_part[(size_t)blk * p.norm + c] = a;
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

// tokens per item, so that a block's rows fill its groups, and heads per
// item: all of a token's heads when there are items enough for every SM four
// times over, else as few as fill the block once (short decode batches).
// Backward a block takes many items, and they are kept to four fillings, so
// that the blocks' shares come out even.
void plan_side(Side* s, int tokens, int rows_in_flight, int num_sms, bool back) {
  if (s->H == 0) {
    s->tile = 1;
    s->hc = 1;
    s->hsplit = 1;
    s->items = 0;
    return;
  }
  s->tile = s->H >= rows_in_flight ? 1 : (rows_in_flight + s->H - 1) / s->H;
  if (s->tile > kTileTokens) s->tile = kTileTokens;
  const int tiles = (tokens + s->tile - 1) / s->tile;
  s->hc = tiles >= 4 * num_sms || s->H < rows_in_flight ? s->H : rows_in_flight;
  if (back && s->hc > 4 * rows_in_flight) s->hc = 4 * rows_in_flight;
  s->hsplit = (s->H + s->hc - 1) / s->hc;
  s->items = tiles * s->hsplit;
}

// blocks of each side in the backward pass: the resident ones shared by rows,
// each side that has rows with at least one
void plan_blocks(NrParams* p, int resident) {
  const long long q = p->side[0].H, k = p->side[1].H;
  for (Side& s : p->side) {
    long long n = s.H == 0 ? 0 : resident * (long long)s.H / (q + k);
    if (s.H > 0 && n < 1) n = 1;
    if (n > s.items) n = s.items;
    s.blocks = (int)n;
  }
}
int lanes_of(int D) { return D <= 64 ? 8 : D <= 640 ? 16 : 32; }
int resident_blocks(int D, int num_sms) {
  return num_sms * (D <= 256 ? bwd_blocks_per_sm<1>() : bwd_blocks_per_sm<4>());
}

template <int G, int V, int MODE>
cudaError_t launch_mode(const LaunchCtx& c, const NrParams& p, bool back) {
  size_t smem = (size_t)kTileTokens * (p.rope / 2) * sizeof(float2);
  if (!back) {
    norm_rope_kernel<G, V, MODE><<<p.side[0].items + p.side[1].items, kThreads, smem, c.stream>>>(p);
  } else {
    const size_t red = (size_t)(kThreads / 32) * G * V * 8 * sizeof(float);
    if (red > smem) smem = red;
    norm_rope_bwd_kernel<G, V, MODE><<<p.side[0].blocks + p.side[1].blocks, kThreads, smem, c.stream>>>(p);
  }
  note_launches(1);
  return cudaGetLastError();
}
// Half-split pairs lie r/2 columns apart: r/16 lanes when that is a power of
// two below G and the rotated range starts on a multiple of r columns.
template <int G, int V>
cudaError_t launch_gv(const LaunchCtx& c, const NrParams& p, bool inter, bool back) {
  if (p.rope == 0) return launch_mode<G, V, kNone>(c, p, back);
  if (inter) return launch_mode<G, V, kInter>(c, p, back);
  const int lanes = p.rope / 16;
  const bool shfl = (lanes & (lanes - 1)) == 0 && lanes < G && (p.D - p.rope) % p.rope == 0;
  return shfl ? launch_mode<G, V, kShfl>(c, p, back) : launch_mode<G, V, kHalf>(c, p, back);
}
cudaError_t launch_nr(const LaunchCtx& c, const NrParams& p, bool inter, bool back) {
  if (p.D <= 64) return launch_gv<8, 1>(c, p, inter, back);
  if (p.D <= 128) return launch_gv<16, 1>(c, p, inter, back);
  if (p.D <= 256) return launch_gv<16, 2>(c, p, inter, back);
  if (p.D <= 640) return launch_gv<16, 5>(c, p, inter, back);
  return launch_gv<32, 4>(c, p, inter, back);
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
  if ((long long)s->B * s->T * (d->Hq + d->Hk) >= (1LL << 31)) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

NrParams make_params(const LaunchCtx& c, const dsa_shape* s, const dsa_norm_rope_desc* d, bool back) {
  NrParams p = {};
  p.map = api_kv_map(s);
  p.inv_freq = d->inv_freq;
  p.tokens = s->B * s->T;
  p.T = s->T;
  p.D = d->D;
  p.norm = d->norm_cols;
  p.rope = d->rope_cols;
  p.inv_norm = d->norm_cols > 0 ? 1.f / (float)d->norm_cols : 0.f;
  p.eps = d->eps;
  p.err = c.err;
  p.side[0].H = d->Hq;
  p.side[1].H = d->Hk;
  p.side[0].w = d->q_weight;
  p.side[1].w = d->k_weight;
  for (Side& sd : p.side) plan_side(&sd, p.tokens, kThreads / lanes_of(d->D), c.num_sms, back);
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
  return ((size_t)resident_blocks(d->D, 256) + 2) * (d->norm_cols > 0 ? d->norm_cols : 1) * sizeof(float);
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
  return launch_nr(c, p, d->interleaved != 0, false) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
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
  plan_blocks(&p, resident_blocks(d->D, c.num_sms));
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
    float* dw[2] = {d->Hq > 0 ? dq_weight : nullptr, d->Hk > 0 ? dk_weight : nullptr};
    for (int i = 0; i < 2; ++i) {
      if (dw[i] == nullptr) continue;
      p.side[i].dw_part = part;
      w.part[i] = part;
      w.dw[i] = dw[i];
      w.blocks[i] = p.side[i].blocks;
      part += (size_t)p.side[i].blocks * p.norm;
    }
  }
  if (launch_nr(c, p, d->interleaved != 0, true) != cudaSuccess) return DSA_ERR_CUDA;
  if (w.dw[0] != nullptr || w.dw[1] != nullptr) {
    norm_rope_dw_kernel<<<dim3((p.norm + 7) / 8, 2), 256, 0, c.stream>>>(w);
    note_launches(1);
    if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  }
  return DSA_OK;
}
