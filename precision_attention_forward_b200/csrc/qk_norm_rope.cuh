// qk_norm_rope.cuh -- per-head RMS norm and multi-axis rotary positions of Q and K in one pass,
// into BF16/FP32 or straight into MXFP8, and the backward pass.
//
// Forward, for a row x of one (token, head), weight w and pair (a, b) of elements:
//   r = rsqrt(mean(x^2) + eps) (1 without the norm),  u = x * r * w,
//   t = position[axis of the pair] * frequency of the pair,
//   y_a = u_a cos t - u_b sin t,  y_b = u_a sin t + u_b cos t.
// Backward, with g the transposed rotation of dy:
//   dw += g * x r,  h = g * w,  dx = r h - x r^3 mean(h x).
// Everything between the loads and the stores is FP32; a value is rounded once, to its output type.
//
// What bounds it: HBM. A row is read once and written once; 16 lanes own a row (8 elements, one
// 16-byte load of BF16 each), so the norm is four shuffles and an interleaved pair never leaves its
// lane; a half pair (i, i + 64) is one shuffle with the lane eight away. A warp has two rows at a
// time and kRopeBatch such pairs of rows in flight. The angles depend on the token alone: a block
// computes those of its few tokens once, into shared memory, and every head of Q and K reads them.
// An angle is a product in FP64 reduced to a fraction of a turn by one FMA (exact up to the
// frequency's own rounding), so far positions keep their accuracy; sincospif does the rest.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "quantize.cuh"

namespace lpfa {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeTile = 8;      // tokens of a forward block (at most)
constexpr int kRopeBwdTile = 32;  // tokens whose angles a backward block holds at a time
constexpr int kRopeBatch = 4;     // rows that a half warp has in flight
// Backward blocks, and with them rows of weight-gradient partials: four for each of 148 SMs.
constexpr int kRopeBwdBlocks = 592;

enum RopeOut : int { kRopeBf16 = 0, kRopeF32 = 1, kRopeMxfp8 = 2 };

// The rotation: frequencies in turns (radians / 2 pi) for a position step of 1, FP64.
struct RopePlan {
  double turns[64];
  uint8_t axis[64];
};

struct RopeTensor {
  const void* x;  // (T, heads, 128), strides in elements
  int64_t tok_stride, head_stride;
  void* out;  // forward: values or MXFP8 payload; backward: dx
  int64_t out_tok, out_head;
  const void* w;  // weight row(s) or NULL (1)
  int64_t w_head;
  uint8_t* scales;  // MXFP8 only
  const void* dy;   // backward only
  int64_t dy_tok, dy_head;
  int heads;  // 0: the tensor is absent
};

struct RopeParams {
  RopeTensor t[2];  // Q, K
  const void* pos;
  int64_t pos_tok, pos_axis;  // elements
  int64_t tokens;
  float eps;
  int pos64;   // positions are int64 (else int32)
  int w_bf16;  // weights are BF16 (else FP32)
  int norm;
  int tile;  // forward: tokens per block; backward: tokens per block in all
  // MXFP8 only
  int num_seqs;
  const int32_t* cu_seqlens;
  const int32_t* scale_off;
  int floor_mode;
  // backward only: [block][rows][128] partial weight gradients, rows = w_rows[0] + w_rows[1]
  float* partials;
  int w_rows[2];  // 0: no weight; 1: one row for all heads; heads: a row each
};

template <typename T>
__device__ __forceinline__ void row_load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void row_load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void row_load8<float>(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// A row's 8 elements as they stand in memory: loaded before anything waits for them. Plain loads
// (not the read-only path): the output may be the input itself.
template <typename T> struct RawRow;
template <> struct RawRow<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
  }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <> struct RawRow<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    a = s[0];
    b = s[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

__device__ __forceinline__ void row_store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]),
                                            cvt_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void row_store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ void weight_load8(const RopeParams& p, const RopeTensor& t, int head, int col, float (&w)[8]) {
  if (t.w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
  } else if (p.w_bf16) {
    row_load8(static_cast<const __nv_bfloat16*>(t.w) + head * t.w_head + col, w);
  } else {
    row_load8(static_cast<const float*>(t.w) + head * t.w_head + col, w);
  }
}

// (cos, sin) of token `tok`, pair `pair`.
__device__ __forceinline__ float2 rope_turn(const RopeParams& p, const RopePlan& plan, int64_t tok, int pair) {
  if (p.pos == nullptr) return make_float2(1.f, 0.f);  // no rotation
  const int64_t at = tok * p.pos_tok + plan.axis[pair] * p.pos_axis;
  const double pos = p.pos64 ? static_cast<double>(__ldg(static_cast<const long long*>(p.pos) + at))
                             : static_cast<double>(__ldg(static_cast<const int*>(p.pos) + at));
  const double f = plan.turns[pair];
  const float frac = static_cast<float>(fma(pos, f, -rint(pos * f)));  // in [-1/2, 1/2] of a turn
  float2 cs;
  sincospif(2.f * frac, &cs.y, &cs.x);
  return cs;
}

// Sum over the 16 lanes of a row; every lane of the warp takes part.
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = 8; m; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v;
}

// Rotates a lane's 8 elements by cs (of the row's token), or back with kBack.
template <bool kHalf, bool kBack>
__device__ __forceinline__ void rotate8(float (&u)[8], const float2* cs, int lane16) {
  if (kHalf) {
    // Elements (i, i + 64): lanes 0..7 hold the first of each pair, lanes 8..15 the second.
    const float4* c4 = reinterpret_cast<const float4*>(cs + (lane16 & 7) * 8);
    const float sign = (lane16 < 8) != kBack ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 c = c4[i];
      const float o0 = __shfl_xor_sync(0xFFFFFFFFu, u[2 * i], 8);
      const float o1 = __shfl_xor_sync(0xFFFFFFFFu, u[2 * i + 1], 8);
      u[2 * i] = fmaf(u[2 * i], c.x, sign * (o0 * c.y));
      u[2 * i + 1] = fmaf(u[2 * i + 1], c.z, sign * (o1 * c.w));
    }
  } else {
    const float4* c4 = reinterpret_cast<const float4*>(cs + lane16 * 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 c = c4[i];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float co = j ? c.z : c.x;
        const float si = kBack ? -(j ? c.w : c.y) : (j ? c.w : c.y);
        const float a = u[4 * i + 2 * j], b = u[4 * i + 2 * j + 1];
        u[4 * i + 2 * j] = fmaf(a, co, -(b * si));
        u[4 * i + 2 * j + 1] = fmaf(a, si, b * co);
      }
    }
  }
}

// Grid: blocks of `tile` tokens (MXFP8: 8 of the 128 rows of a padded block: rows r0, r0 + 1 of each
// 32-row quarter, which together fill whole sectors of the scale atoms). TIn, kOut, kHalf as named.
template <typename TIn, int kOut, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads)
qk_norm_rope_kernel(const __grid_constant__ RopeParams p, const __grid_constant__ RopePlan plan) {
  __shared__ __align__(16) float2 cs[kRopeTile][64];
  __shared__ int64_t tok_of[kRopeTile];  // -1: no such token
  extern __shared__ __align__(16) uint32_t sf_words[];  // MXFP8: [Q and K head][8 rows], the rows' four scale bytes
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = lane >> 4, l16 = lane & 15;
  int64_t atom0 = 0;  // MXFP8: 128-token block, and the first row of this tile in its quarter
  int r0 = 0;
  const int ntok = kOut == kRopeMxfp8 ? kRopeTile : p.tile;

  if (kOut == kRopeMxfp8) {
    atom0 = blockIdx.x >> 4;
    r0 = (blockIdx.x & 15) * 2;
    if (threadIdx.x < kRopeTile) {
      const int seq = find_seq(p.scale_off, p.num_seqs, static_cast<int>(atom0));
      const int start = __ldg(p.cu_seqlens + seq);
      const int64_t in_seq = (atom0 - __ldg(p.scale_off + seq)) * 128 + r0 + (threadIdx.x & 1) + 32 * (threadIdx.x >> 1);
      tok_of[threadIdx.x] = in_seq < __ldg(p.cu_seqlens + seq + 1) - start ? start + in_seq : -1;
    }
  } else if (threadIdx.x < ntok) {
    const int64_t tok = static_cast<int64_t>(blockIdx.x) * ntok + threadIdx.x;
    tok_of[threadIdx.x] = tok < p.tokens ? tok : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < ntok * 64; i += kRopeThreads) {
    const int64_t tok = tok_of[i >> 6];
    if (tok >= 0) cs[i >> 6][i & 63] = rope_turn(p, plan, tok, i & 63);
  }
  __syncthreads();

#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const RopeTensor& t = p.t[which];
    if (t.heads == 0) continue;
    const int rows = ntok * t.heads;
    const float per_head = 1.f / static_cast<float>(t.heads);
    float w[8];
    weight_load8(p, t, 0, l16 * 8, w);
#pragma unroll 1
    for (int base = 2 * warp; base < rows; base += 2 * kRopeWarps * kRopeBatch) {
      RawRow<TIn> raw[kRopeBatch];
      int64_t tok[kRopeBatch];
      int slot[kRopeBatch], head[kRopeBatch];
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        const int r = base + 2 * kRopeWarps * u + half;
        // r / heads: r + 1/2 keeps the product off the whole numbers (r < 2^16).
        slot[u] = static_cast<int>((static_cast<float>(r) + 0.5f) * per_head);
        head[u] = r - slot[u] * t.heads;
        tok[u] = r < rows ? tok_of[slot[u]] : -2;  // -2: beyond the tile, -1: a padding row
        if (tok[u] >= 0)
          raw[u].load(t.x, tok[u] * t.tok_stride + head[u] * t.head_stride + l16 * 8);
        else
          raw[u].zero();
      }
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        if (base + 2 * kRopeWarps * u >= rows) break;  // the same for the whole warp
        float v[8];
        raw[u].get(v);
        if (p.norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
          const float r = rsqrtf(row_sum(ss) * (1.f / 128.f) + p.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= r;
        }
        if (t.w_head != 0) weight_load8(p, t, head[u], l16 * 8, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= w[i];
        rotate8<kHalf, false>(v, cs[tok[u] >= 0 ? slot[u] : 0], l16);
        if (kOut == kRopeMxfp8) {
          // The quantizer's rule (quantize.cuh): a 32-element block is four lanes.
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
          amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
          const int e = e8m0_exponent(amax, p.floor_mode);
          const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          if (tok[u] >= 0) {
            const uint32_t w0 = cvt_e4m3x2(v[0] * inv, v[1] * inv) |
                                (static_cast<uint32_t>(cvt_e4m3x2(v[2] * inv, v[3] * inv)) << 16);
            const uint32_t w1 = cvt_e4m3x2(v[4] * inv, v[5] * inv) |
                                (static_cast<uint32_t>(cvt_e4m3x2(v[6] * inv, v[7] * inv)) << 16);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.out) + (tok[u] * t.heads + head[u]) * 128 + l16 * 8) =
                make_uint2(w0, w1);
          }
          if (tok[u] >= -1 && (l16 & 3) == 0)
            reinterpret_cast<uint8_t*>(sf_words + ((which ? p.t[0].heads : 0) + head[u]) * kRopeTile +
                                       (slot[u] & 1) * 4 + (slot[u] >> 1))[l16 >> 2] =
                tok[u] >= 0 ? static_cast<uint8_t>(e + 127) : uint8_t{0x7F};
        } else if (tok[u] >= 0) {
          const int64_t at = tok[u] * t.out_tok + head[u] * t.out_head + l16 * 8;
          if (kOut == kRopeBf16)
            row_store8(static_cast<__nv_bfloat16*>(t.out) + at, v);
          else
            row_store8(static_cast<float*>(t.out) + at, v);
        }
      }
    }
  }
  if (kOut == kRopeMxfp8) {
    // Row r0 + j of the four quarters: 16 contiguous bytes of the head's atom.
    __syncthreads();
    const int hq = p.t[0].heads;
    for (int i = threadIdx.x; i < 2 * (hq + p.t[1].heads); i += kRopeThreads) {
      const int row = i & 1, h = i >> 1;
      const RopeTensor& t = p.t[h >= hq];
      const int head = h >= hq ? h - hq : h;
      *reinterpret_cast<uint4*>(t.scales + (atom0 * t.heads + head) * 512 + (r0 + row) * 16) =
          *reinterpret_cast<const uint4*>(sf_words + h * kRopeTile + row * 4);
    }
  }
}

// Backward. Each block walks `tile` consecutive tokens, kRopeBwdTile at a time. A half warp keeps
// one head while it walks tokens, so the weight gradient of its 8 channels stays in registers: one
// sum over everything it saw (one weight row), or one per head, added to the block's own row of
// partials. No atomics: the same sums in the same order every time.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads)
qk_norm_rope_bwd_kernel(const __grid_constant__ RopeParams p, const __grid_constant__ RopePlan plan) {
  constexpr int kHalves = 2 * kRopeWarps;
  constexpr int kBatch = 2;
  __shared__ __align__(16) float2 cs[kRopeBwdTile][64];
  __shared__ __align__(16) float sums[kHalves][128];
  const int lane = threadIdx.x & 31, l16 = lane & 15;
  const int hw = threadIdx.x >> 4;  // half warp
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.tile;
  const int64_t last = min(first + p.tile, p.tokens);
  const int part_rows = p.w_rows[0] + p.w_rows[1];
  float* part = p.partials + static_cast<int64_t>(blockIdx.x) * part_rows * 128;

  float acc[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0.f;

  for (int64_t tok0 = first; tok0 < last; tok0 += kRopeBwdTile) {
    const int ntok = static_cast<int>(min(static_cast<int64_t>(kRopeBwdTile), last - tok0));
    __syncthreads();  // the angles of the previous tokens have been read
    for (int i = threadIdx.x; i < ntok * 64; i += kRopeThreads)
      cs[i >> 6][i & 63] = rope_turn(p, plan, tok0 + (i >> 6), i & 63);
    __syncthreads();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const RopeTensor& t = p.t[which];
      const bool per_head = p.w_rows[which] > 1;
#pragma unroll 1
      for (int h0 = 0; h0 < t.heads; h0 += kHalves) {
        // nh heads on the half warps, `groups` half warps sharing the tokens of each.
        const int nh = min(kHalves, t.heads - h0);
        const int groups = kHalves / nh;
        const int grp = hw / nh;
        const int head = h0 + hw - grp * nh;
        float w[8];
        weight_load8(p, t, t.w_head ? head : 0, l16 * 8, w);
#pragma unroll 1
        for (int s0 = 0; s0 < ntok; s0 += kBatch * groups) {
          RawRow<T> rx[kBatch], rd[kBatch];
          bool on[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int s = s0 + u * groups + grp;
            on[u] = grp < groups && s < ntok;
            if (on[u]) {
              rx[u].load(t.x, (tok0 + s) * t.tok_stride + head * t.head_stride + l16 * 8);
              rd[u].load(t.dy, (tok0 + s) * t.dy_tok + head * t.dy_head + l16 * 8);
            } else {
              rx[u].zero();
              rd[u].zero();
            }
          }
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int s = s0 + u * groups + grp;
            float x[8], g[8];
            rx[u].get(x);
            rd[u].get(g);
            rotate8<kHalf, true>(g, cs[on[u] ? s : 0], l16);
            float r = 1.f, m = 0.f;
            if (p.norm) {
              float ss = 0.f, hx = 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                ss = fmaf(x[i], x[i], ss);
                hx = fmaf(g[i] * w[i], x[i], hx);
              }
              ss = row_sum(ss);
              hx = row_sum(hx);
              r = rsqrtf(ss * (1.f / 128.f) + p.eps);
              m = hx * (1.f / 128.f) * r * r;
            }
            float dx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              dx[i] = r * (g[i] * w[i] - x[i] * m);
              acc[which][i] = fmaf(g[i], x[i] * r, acc[which][i]);  // zero rows add nothing
            }
            if (on[u]) row_store8(static_cast<T*>(t.out) + (tok0 + s) * t.out_tok + head * t.out_head + l16 * 8, dx);
          }
        }
        if (per_head) {
          // The block's sum for these heads, over the half warps that shared each.
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            sums[hw][l16 * 8 + i] = acc[which][i];
            acc[which][i] = 0.f;
          }
          __syncthreads();
          for (int i = threadIdx.x; i < nh * 128; i += kRopeThreads) {
            float s = 0.f;
            for (int g = 0; g < groups; ++g) s += sums[g * nh + (i >> 7)][i & 127];
            float* to = part + (which * p.w_rows[0] + h0) * 128 + i;
            *to = tok0 == first ? s : *to + s;
          }
          __syncthreads();
        }
      }
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (p.w_rows[which] != 1) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[hw][l16 * 8 + i] = acc[which][i];
    __syncthreads();
    if (threadIdx.x < 128) {
      float s = 0.f;
      for (int g = 0; g < kHalves; ++g) s += sums[g][threadIdx.x];
      part[which * p.w_rows[0] * 128 + threadIdx.x] = s;
    }
  }
}

// Sums the blocks' partial weight gradients: one block of 8 x 128 threads for a row of the result.
__global__ void __launch_bounds__(1024)
qk_norm_rope_dw_kernel(const float* partials, int blocks, int rows, int rows_q, float* dwq, float* dwk) {
  __shared__ float sums[8][128];
  const int row = blockIdx.x, ch = threadIdx.x & 127, grp = threadIdx.x >> 7;
  float s = 0.f;
#pragma unroll 8
  for (int b = grp; b < blocks; b += 8) s += __ldg(partials + (static_cast<int64_t>(b) * rows + row) * 128 + ch);
  sums[grp][ch] = s;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int g = 1; g < 8; ++g) s += sums[g][ch];
    (row < rows_q ? dwq + row * 128 : dwk + (row - rows_q) * 128)[ch] = s;
  }
}

}  // namespace lpfa
