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
// What bounds it: HBM, once the arithmetic is out of the way (a first version with one element per
// FP32 instruction and 16 lanes per row needed 79 warp instructions per row and took 191 us for 32768
// tokens x 48 heads of BF16). So eight lanes own a row: a lane has elements 8 j .. 8 j + 7 and 64 + 8 j
// .. 64 + 8 j + 7, whole 16-byte pieces that hold complete pairs of either pairing, and the arithmetic
// is on two floats at a time (f32x2). A warp takes four rows in a step and two steps together, so that
// their chains of shuffles and conversions overlap, and has the next two on their way in shared memory.
// The weight is folded into the rotation (w_a cos, w_b sin, ...) once per token, for all heads. The
// angles depend on the token alone: a warp computes its token's once. An angle is a product in FP64
// reduced by one FMA to a rest of at most an eighth of a turn (exact up to the frequency's own
// rounding), so far positions keep their accuracy, and short series do the rest.
// Measured (B200): that case 127 us, the time of a device copy of its bytes; 8192 tokens x 32 heads of
// BF16 into MXFP8 29 us, bound by the latency of shuffles and conversions at 16 warps an SM: its 270 warp
// instructions a step (4 rows: norm and rotation 150, block maxima, scale bytes and conversion 120) take 56 % of
// the issue slots; ragged FP32 sequences into MXFP8 at 95 % of the copy
// bandwidth, and at 85 % once the power limit has lowered the clock.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "quantize.cuh"

namespace lpfa {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeTokens = 4 * kRopeWarps;  // tokens of a forward block, at most
constexpr int kRopeBatch = 2;                // forward steps that a warp takes together
// Batches of a warp's shared-memory ring (2 KB each for BF16 input, 4 KB for FP32): one computed, one on
// the way. More of them are slower: with four (three) the video forward took 151 us when it took 132 with two,
// and the ragged FP32 to MXFP8 one 272 against 258, since the warps' tokens lie apart in memory and
// each keeps more places of it open.
template <typename T> constexpr int rope_stages() { return 2; }
template <typename T> constexpr int rope_stage_bytes() { return kRopeBatch * 4 * 128 * static_cast<int>(sizeof(T)); }
template <typename T> constexpr int rope_smem_bytes() {
  return kRopeTokens * 64 * 8 + kRopeWarps * rope_stages<T>() * rope_stage_bytes<T>();
}
constexpr int kRopeBwdTile = 64;             // tokens whose angles a backward block holds at a time
// Backward blocks, and with them rows of weight-gradient partials: two for each of 148 SMs.
constexpr int kRopeBwdBlocks = 296;

template <typename T> constexpr int rope_bwd_stage() { return 2 * 4 * 128 * static_cast<int>(sizeof(T)); }
template <typename T> constexpr int rope_bwd_smem() {
  return kRopeBwdTile * 128 * 4 + 4 * kRopeWarps * 128 * 4 + kRopeWarps * 2 * rope_bwd_stage<T>();
}

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
  int quad;  // 1: a warp's four rows are heads of one token; 0: the same head of four tokens
  int items, whole, parts;  // forward: items of work; tiles that are one item each; parts of each of the others
  int batches;              // forward: batches of steps of such a part
  int tile;                 // backward: tokens per block in all
  // MXFP8 only
  int num_seqs;
  const int32_t* cu_seqlens;
  const int32_t* scale_off;
  int floor_mode;
  // backward only: [block][rows][128] partial weight gradients, rows = w_rows[0] + w_rows[1]
  float* partials;
  int w_rows[2];  // 0: no weight; 1: one row for all heads; heads: a row each
};

// Two floats in one register pair, and the arithmetic on them.
typedef float2 F2;
__device__ __forceinline__ F2 f2(float lo, float hi) { return make_float2(lo, hi); }
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float f2_sum(F2 a) { return a.x + a.y; }
__device__ __forceinline__ void f2_get(F2 a, float& lo, float& hi) {
  lo = a.x;
  hi = a.y;
}
// max(a, |b|, |c|) for a >= 0, and max over a chunk's 8 magnitudes.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float chunk_amax(const float (&v)[8]) {
  float m = max3_abs(v[0], v[1], v[2]);
  m = max3_abs(m, v[3], v[4]);
  m = max3_abs(m, v[5], v[6]);
  return fmaxf(m, fabsf(v[7]));
}

// Scale byte for a block maximum, the bits of e8m0_exponent(amax, floor_mode) + 127: `up` carries a
// mantissa above 1.75 into the exponent (RCEIL) or is 0 (FLOOR); 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t e4m3_scale_byte(float amax, uint32_t up) {
  return max((__float_as_uint(amax) + up) >> 23, 8u) - 8u;
}
constexpr uint32_t kE4m3Up = 0x1FFFFFu;

// Four floats -> four E4M3 codes (round to nearest even, saturate to +-448).
__device__ __forceinline__ uint32_t cvt_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void lds16(uint4& v, uint32_t at) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
}

// A lane's 16 elements of a row as they stand in memory (chunks at 8 j and 64 + 8 j): loaded before
// anything waits for them. Plain loads, not the read-only path: the output may be the input itself.
template <typename T> struct RawRow;
template <> struct RawRow<__nv_bfloat16> {
  uint4 c[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    c[0] = *reinterpret_cast<const uint4*>(p);
    c[1] = *reinterpret_cast<const uint4*>(p + 64);
  }
  __device__ __forceinline__ void load_shared(uint32_t at, int lane) {
    lds16(c[0], at + lane * 16);
    lds16(c[1], at + 512 + lane * 16);
  }
  __device__ __forceinline__ void get(int k, float (&v)[8]) const {
    const uint32_t w[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <> struct RawRow<float> {
  float4 c[4];
  __device__ __forceinline__ void load(const float* p) {
    const float4* s = reinterpret_cast<const float4*>(p);
    c[0] = s[0];
    c[1] = s[1];
    c[2] = s[16];
    c[3] = s[17];
  }
  // (pieces 2 j, 2 j + 1, 16 + 2 j, 17 + 2 j of the row, where those of odd runs have changed places)
  __device__ __forceinline__ void load_shared(uint32_t at, int lane) {
    const int j = lane & 7;
    at += (lane >> 3) * 512;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 u;
      const int piece = (i >> 1) * 16 + 2 * j + (i & 1);
      lds16(u, at + (piece ^ ((piece >> 3) & 1)) * 16);
      c[i] = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
    }
  }
  __device__ __forceinline__ void get(int k, float (&v)[8]) const {
    const float4 a = c[2 * k], b = c[2 * k + 1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// Copies four rows of a warp (lane: its row's element 8 j, FP32: 4 j) to shared memory, for load_shared:
// whole 128-byte runs of a row, and for FP32 with the pieces of odd runs exchanged, so that
// load_shared's reads are free of bank conflicts.
__device__ __forceinline__ void row_async(uint32_t dst, const __nv_bfloat16* p, int lane) {
  cp_async16(dst + lane * 16, p, 16);
  cp_async16(dst + 512 + lane * 16, p + 64, 16);
}
__device__ __forceinline__ void row_async(uint32_t dst, const float* p, int lane) {
  const int j = lane & 7;
#pragma unroll
  for (int c = 0; c < 4; ++c) cp_async16(dst + (lane >> 3) * 512 + (c * 8 + (j ^ (c & 1))) * 16, p + 32 * c, 16);
}

// The same 16 elements as eight pairs: a[i] holds the first elements of pairs 2 i and 2 i + 1, b[i]
// the second ones. Pairs: interleaved 4 j .. 4 j + 3 and 32 + 4 j .. 32 + 4 j + 3; half 8 j .. 8 j + 7.
struct Pairs {
  F2 a[4], b[4];
};

// Lane j's pairs 0 .. 7 are pairs 8 j .. 8 j + 7 of the head (half), or 4 j .. 4 j + 3 and 32 on (interleaved).
// A token's angles lie in shared memory as the lanes take them: cos and sin of pairs 2 i and 2 i + 1 of lane
// j are the four floats at 4 (8 i + j), so that eight lanes read 128 bytes in a row and find two pairs
// side by side (in the order of the pairs, with bank conflicts, the backward pass that takes 43.4 us took
// 45.0). turn_word: the word of pair p's cos; its sin is two further.
template <bool kHalf>
__device__ __forceinline__ int turn_word(int p) {
  const int j = kHalf ? p >> 3 : (p & 31) >> 2;
  const int i = kHalf ? p & 7 : (p & 3) + 4 * (p >> 5);
  return 4 * (8 * (i >> 1) + j) + (i & 1);
}

template <bool kHalf>
__device__ __forceinline__ Pairs to_pairs(const float (&x)[8], const float (&y)[8]) {  // chunks at 8 j, 64 + 8 j
  Pairs p;
  if (kHalf) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p.a[i] = f2(x[2 * i], x[2 * i + 1]);
      p.b[i] = f2(y[2 * i], y[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      p.a[i] = f2(x[4 * i], x[4 * i + 2]);
      p.b[i] = f2(x[4 * i + 1], x[4 * i + 3]);
      p.a[2 + i] = f2(y[4 * i], y[4 * i + 2]);
      p.b[2 + i] = f2(y[4 * i + 1], y[4 * i + 3]);
    }
  }
  return p;
}

template <bool kHalf>
__device__ __forceinline__ void from_pairs(const Pairs& p, float (&x)[8], float (&y)[8]) {
  if (kHalf) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f2_get(p.a[i], x[2 * i], x[2 * i + 1]);
      f2_get(p.b[i], y[2 * i], y[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f2_get(p.a[i], x[4 * i], x[4 * i + 2]);
      f2_get(p.b[i], x[4 * i + 1], x[4 * i + 3]);
      f2_get(p.a[2 + i], y[4 * i], y[4 * i + 2]);
      f2_get(p.b[2 + i], y[4 * i + 1], y[4 * i + 3]);
    }
  }
}

__device__ __forceinline__ void chunk_store(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]),
                                            cvt_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void chunk_store(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <bool kHalf>
__device__ __forceinline__ Pairs weight_pairs(const RopeParams& p, const RopeTensor& t, int head, int j) {
  float x[8], y[8];
  if (t.w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 1.f;
  } else if (p.w_bf16) {
    RawRow<__nv_bfloat16> r;
    r.load(static_cast<const __nv_bfloat16*>(t.w) + head * t.w_head + 8 * j);
    r.get(0, x);
    r.get(1, y);
  } else {
    RawRow<float> r;
    r.load(static_cast<const float*>(t.w) + head * t.w_head + 8 * j);
    r.get(0, x);
    r.get(1, y);
  }
  return to_pairs<kHalf>(x, y);
}

// The rotations that a lane computes, those of pairs `lane` and `lane + 32`: read once (a lane's own
// entries of the kernel's constants are a serialised read, 13 us of the video forward when it was
// done for every token).
struct LaneTurns {
  double f[2];
  int64_t axis[2];  // offsets in the position row
};
__device__ __forceinline__ LaneTurns lane_turns(const RopeParams& p, const RopePlan& plan, int lane) {
  LaneTurns r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r.f[i] = plan.turns[lane + 32 * i];
    r.axis[i] = plan.axis[lane + 32 * i] * p.pos_axis;
  }
  return r;
}

__device__ __forceinline__ int64_t rope_position(const RopeParams& p, int64_t at) {
  if (p.pos == nullptr) return 0;
  return p.pos64 ? __ldg(static_cast<const long long*>(p.pos) + at) : __ldg(static_cast<const int*>(p.pos) + at);
}

// (cos, sin) of position n at f turns a step.
__device__ __forceinline__ float2 rope_turn(int64_t n, double f) {
  const double pos = static_cast<double>(n);
  // Quarter turns, and a rest in [-1/8, 1/8] of a turn whose FP32 rounding is below 2^-28.
  const double quarters = rint(pos * f * 4.0);
  const float rest = static_cast<float>(fma(pos, f, -0.25 * quarters));
  // sin and cos of at most pi / 4: the Taylor series to x^9 and x^10 (the next terms are below 2^-29).
  const float x = 6.28318530718f * rest, x2 = x * x;
  float s = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
  s = fmaf(x2, s, 1.f / 120.f);
  s = fmaf(x2, s, -1.f / 6.f);
  s = fmaf(x * x2, s, x);
  float c = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
  c = fmaf(x2, c, -1.f / 720.f);
  c = fmaf(x2, c, 1.f / 24.f);
  c = fmaf(x2, c, -0.5f);
  c = fmaf(x2, c, 1.f);
  const int q = static_cast<int>(static_cast<long long>(quarters)) & 3;
  const float co = (q & 1) ? s : c, si = (q & 1) ? c : s;
  return make_float2((q == 1 || q == 2) ? -co : co, q >= 2 ? -si : si);
}

// 1 / sqrt(v): the approximation and one Newton step.
__device__ __forceinline__ float rsqrt_newton(float v) {
  const float r = rsqrtf(v);
  const float e = fmaf(-v * r, r, 1.f);
  return e == e ? fmaf(0.5f * r, e, r) : r;  // (0 and infinity: r is right as it is)
}

// Sum over the 8 lanes of a row; every lane of the warp takes part.
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = 4; m; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v;
}

template <bool kHalf>
__device__ __forceinline__ void put_turn(float* cs, int pair, float2 turn) {
  float* to = cs + turn_word<kHalf>(pair);
  to[0] = turn.x;
  to[2] = turn.y;
}

// cos and sin of lane j's pairs.
__device__ __forceinline__ void turn_pairs(const float* cs, int j, F2 (&c)[4], F2 (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(cs + 4 * (8 * i + j));
    c[i] = f2(v.x, v.y);
    s[i] = f2(v.z, v.w);
  }
}

// The rotation with the weight in it: y_a = x_a ac + x_b bs, y_b = x_a as + x_b bc.
struct Turn {
  F2 ac[4], bs[4], as[4], bc[4];
};
template <bool kHalf>
__device__ __forceinline__ void make_turn(Turn& m, const float* cs, const Pairs& w, int j) {
  const F2 minus = f2(-1.f, -1.f);
  F2 c[4], s[4];
  turn_pairs(cs, j, c, s);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m.ac[i] = f2_mul(w.a[i], c[i]);
    m.as[i] = f2_mul(w.a[i], s[i]);
    m.bc[i] = f2_mul(w.b[i], c[i]);
    m.bs[i] = f2_mul(f2_mul(w.b[i], s[i]), minus);
  }
}

// A warp's four rows are four heads of one token (quad) or, where the head counts are not multiples of four,
// one head of four tokens; a step is four rows, and an item the batches of Q's steps and then K's of
// a tile of tokens. Items go round the blocks. The tiles left after the last whole round (all of them, in
// a small call) are split by heads into p.parts items of p.batches batches each, as many as fill the
// round: 8192 tokens x 32 heads into MXFP8, where 136 of 1024 tiles are left, took 32.8 us with whole tiles and
// 30.8 with halves. A tile is 8 (32) tokens: consecutive ones, or for MXFP8 the rows r0, r0 + 1
// (.. r0 + 7) of each 32-row quarter of a padded 128-token block, whose scale words fill whole sectors
// of the atoms between them. The warps are on their own, without a barrier: each computes its tokens'
// angles while its first rows are on the way, and loads ahead into its next token. (The other mapping, in
// which a block's warps share each token's rows and sweep contiguous memory, needs a barrier and an
// address calculation per item: 167 us when the video forward took 132.)
template <typename TIn, int kOut, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads, 2)
qk_norm_rope_kernel(const __grid_constant__ RopeParams p, const __grid_constant__ RopePlan plan) {
  constexpr int kBatch = kRopeBatch;
  constexpr int kStages = rope_stages<TIn>();
  constexpr int kStageBytes = rope_stage_bytes<TIn>();
  extern __shared__ __align__(16) uint8_t rope_smem[];
  float(*cs)[128] = reinterpret_cast<float(*)[128]>(rope_smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane >> 3, j = lane & 7;
  const int ntok = p.quad ? kRopeWarps : kRopeTokens;
  const int slot = p.quad ? warp : warp * 4 + grp;  // this lane's token of a tile
  const int span = ntok / 4;                        // MXFP8: rows of a quarter
  const int parts = 32 / span;                      // MXFP8: tiles of a 128-token block
  const int in_block = slot % span + 32 * (slot / span);
  const float* my_cs = cs[slot];

  struct Place {
    int tok;         // token; 0 where there is none (read the first, write nothing)
    int block, row;  // MXFP8: 128-token block, and the row in it
    bool real;
  };
  auto place = [&](int tile) {
    Place w;
    w.block = 0;
    w.row = 0;
    if (kOut == kRopeMxfp8) {
      w.block = tile / parts;
      w.row = (tile % parts) * span + in_block;
      const int seq = find_seq(p.scale_off, p.num_seqs, w.block);
      const int start = __ldg(p.cu_seqlens + seq);
      const int64_t in_seq = static_cast<int64_t>(w.block - __ldg(p.scale_off + seq)) * 128 + w.row;
      w.tok = static_cast<int>(start + in_seq);
      w.real = in_seq < __ldg(p.cu_seqlens + seq + 1) - start;
    } else {
      const int64_t tok = static_cast<int64_t>(tile) * ntok + slot;
      w.tok = static_cast<int>(tok);
      w.real = tok < p.tokens;
    }
    if (!w.real) w.tok = 0;
    return w;
  };

  const int heads_per_step = p.quad ? 4 : 1;
  const int head0 = p.quad ? grp : 0;  // of this lane's row within a step
  // Batches of kBatch steps, Q's first, then K's; the last one of a tensor may have one step only.
  // (quad: the heads of both are multiples of four)
  const int steps_of[2] = {p.t[0].heads / heads_per_step, p.t[1].heads / heads_per_step};
  const int batches_q = (steps_of[0] + kBatch - 1) / kBatch;
  const int batches = batches_q + (steps_of[1] + kBatch - 1) / kBatch;
  struct Item {
    int tile, b0, b1;  // batches b0 .. b1 of a tile
  };
  auto item_at = [&](int n) {
    Item it = {n, 0, batches};
    if (n >= p.whole) {
      const int part = (n - p.whole) % p.parts;
      it.tile = p.whole + (n - p.whole) / p.parts;
      it.b0 = part * p.batches;
      it.b1 = min(it.b0 + p.batches, batches);
    }
    return it;
  };

  // The loads run ahead, batch after batch and tile after tile, into the warp's ring.
  const uint32_t ring = smem_u32(rope_smem) + kRopeTokens * 64 * 8 + warp * kStages * kStageBytes;
  constexpr int kLaneElems = sizeof(TIn) == 2 ? 8 : 4;  // elements of a copy
  int rd_item = blockIdx.x, rd_batch = 0, rd_end = 0, rd_left = 0;
  bool rd_first = false;
  uint32_t rd_stage = 0;
  Place rd_place = {}, coming = {};  // where the loads are; of the tile whose first batch was loaded last
  int64_t rd_step = 0;
  const TIn* rd = nullptr;
  auto rd_enter = [&](int which, int step) {
    const RopeTensor& t = p.t[which];
    rd = static_cast<const TIn*>(t.x) + rd_place.tok * t.tok_stride + (step * heads_per_step + head0) * t.head_stride + kLaneElems * j;
    rd_step = heads_per_step * t.head_stride;
    rd_left = steps_of[which] - step;
  };
  auto rd_start = [&]() {
    const Item it = item_at(rd_item);
    rd_place = place(it.tile);
    rd_batch = it.b0;
    rd_end = it.b1;
    rd_first = true;
    if (it.b0 < batches_q) rd_enter(0, it.b0 * kBatch); else rd_enter(1, (it.b0 - batches_q) * kBatch);
  };
  auto issue = [&]() {
    if (rd_item < p.items) {
      if (rd_first) coming = rd_place;
      rd_first = false;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (u < rd_left) {
          const uint32_t dst = ring + rd_stage + u * (kStageBytes / kBatch);
          row_async(dst, rd, lane);
          rd += rd_step;
        }
      }
      rd_left -= kBatch;
      rd_stage = rd_stage + kStageBytes == kStages * kStageBytes ? 0 : rd_stage + kStageBytes;
      if (++rd_batch == rd_end) {
        rd_item += gridDim.x;
        if (rd_item < p.items) rd_start();
      } else if (rd_batch == batches_q) {
        rd_enter(1, 0);
      }
    }
    cp_async_commit();
  };
  const uint32_t up = p.floor_mode ? 0u : kE4m3Up;
  if (rd_item >= p.items) return;
  rd_start();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue();
  const LaneTurns turns = lane_turns(p, plan, lane);
  uint32_t stage = 0;
  auto take = [&](RawRow<TIn> (&raw)[kBatch]) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) raw[u].load_shared(ring + stage + u * (kStageBytes / kBatch), lane);
    stage = stage + kStageBytes == kStages * kStageBytes ? 0 : stage + kStageBytes;
  };

#pragma unroll 1
  for (int n = blockIdx.x; n < p.items; n += gridDim.x) {
    static_assert(kStages == 2, "the loads are one batch ahead: in this item, then in the next one's first");
    const Place now = coming;
    const Item it = item_at(n);
    const int b0 = it.b0, b1 = it.b1;
    // The angles of the warp's tokens.
    __syncwarp();  // the previous ones have been read
#pragma unroll 1
    for (int of = 0; of < (p.quad ? 1 : 4); ++of) {
      const int at = __shfl_sync(0xFFFFFFFFu, now.tok, of * 8);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        put_turn<kHalf>(cs[(p.quad ? warp : warp * 4) + of], lane + 32 * i,
                        rope_turn(rope_position(p, at * p.pos_tok + turns.axis[i]), turns.f[i]));
    }
    __syncwarp();

    // The tensor that the steps have come to.
    Turn m;
    int head = 0;
    bool per_head = false;
    uint8_t *sf = nullptr, *bytes = nullptr;
    __nv_bfloat16* out16 = nullptr;
    float* out32 = nullptr;
    int64_t out_step = 0;
    auto enter = [&](int which, int step) {
      const RopeTensor& t = p.t[which];
      const Pairs w = weight_pairs<kHalf>(p, t, 0, j);
      make_turn<kHalf>(m, my_cs, w, j);
      per_head = t.w_head != 0;
      head = step * heads_per_step + head0;
      // Where this lane's row goes: values, or payload bytes and its scale bytes.
      if (kOut == kRopeMxfp8) {
        sf = t.scales + (static_cast<int64_t>(now.block) * t.heads + head) * 512 + (now.row & 31) * 16 + (now.row >> 5) * 4;
        bytes = static_cast<uint8_t*>(t.out) + (static_cast<int64_t>(now.tok) * t.heads + head) * 128 + 8 * j;
      } else if (kOut == kRopeBf16) {
        out16 = static_cast<__nv_bfloat16*>(t.out) + now.tok * t.out_tok + head * t.out_head + 8 * j;
      } else {
        out32 = static_cast<float*>(t.out) + now.tok * t.out_tok + head * t.out_head + 8 * j;
      }
      out_step = heads_per_step * t.out_head;
    };
    if (b0 < batches_q) enter(0, b0 * kBatch); else enter(1, (b0 - batches_q) * kBatch);
    // One batch. The steps of a batch have nothing between them, so that their chains of shuffles
    // and conversions overlap; a step that does not exist is computed and not stored.
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      cp_async_wait<kStages - 2>();
      if (sizeof(TIn) == 4) __syncwarp();  // (BF16: every lane reads what it copied itself)
      RawRow<TIn> raw[kBatch];
      take(raw);
      issue();  // into the stage that the previous batch was taken from
      const bool is_k = b >= batches_q;
      if (b == batches_q && b != b0) enter(1, 0);
      const int left = steps_of[is_k] - (is_k ? b - batches_q : b) * kBatch;
      float x[kBatch][8], y[kBatch][8];
      Pairs v[kBatch];
      F2 r[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        raw[u].get(0, x[u]);
        raw[u].get(1, y[u]);
        v[u] = to_pairs<kHalf>(x[u], y[u]);
        r[u] = f2(1.f, 1.f);
      }
      if (p.norm) {
        float sum[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          F2 ss = f2_mul(v[u].a[0], v[u].a[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) ss = f2_fma(v[u].a[i], v[u].a[i], ss);
#pragma unroll
          for (int i = 0; i < 4; ++i) ss = f2_fma(v[u].b[i], v[u].b[i], ss);
          sum[u] = f2_sum(ss);
        }
#pragma unroll
        for (int k = 4; k; k >>= 1)
#pragma unroll
          for (int u = 0; u < kBatch; ++u) sum[u] += __shfl_xor_sync(0xFFFFFFFFu, sum[u], k);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const float inv = rsqrt_newton(sum[u] * (1.f / 128.f) + p.eps);
          r[u] = f2(inv, inv);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (per_head) {
          const Pairs w = weight_pairs<kHalf>(p, p.t[is_k], u < left ? head + u * heads_per_step : head, j);
          make_turn<kHalf>(m, my_cs, w, j);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 a = f2_mul(v[u].a[i], r[u]), b = f2_mul(v[u].b[i], r[u]);
          v[u].a[i] = f2_fma(a, m.ac[i], f2_mul(b, m.bs[i]));
          v[u].b[i] = f2_fma(a, m.as[i], f2_mul(b, m.bc[i]));
        }
        from_pairs<kHalf>(v[u], x[u], y[u]);
      }
      if (kOut == kRopeMxfp8) {
        // The quantizer's rule (quantize.cuh): a 32-element block is a chunk of four lanes.
        float amax[kBatch][2];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          amax[u][0] = chunk_amax(x[u]);
          amax[u][1] = chunk_amax(y[u]);
        }
#pragma unroll
        for (int k = 1; k < 4; k <<= 1)
#pragma unroll
          for (int u = 0; u < kBatch; ++u)
#pragma unroll
            for (int c = 0; c < 2; ++c) amax[u][c] = fmaxf(amax[u][c], __shfl_xor_sync(0xFFFFFFFFu, amax[u][c], k));
        uint32_t sfw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const uint32_t lo = e4m3_scale_byte(amax[u][0], up), hi = e4m3_scale_byte(amax[u][1], up);
          sfw[u] = lo | (hi << 16);
        }
        // Blocks 0, 2 are lanes 0 .. 3's, 1, 3 lanes 4 .. 7's.
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const uint32_t mine = sfw[u];
          sfw[u] |= __shfl_xor_sync(0xFFFFFFFFu, mine, 4) << 8;
          if (j == 0 && u < left) *reinterpret_cast<uint32_t*>(sf) = now.real ? sfw[u] : 0x7F7F7F7Fu;
          // Scaled as pairs, which is how they stand in the registers: chunk 0 is a and b of pairs 0 .. 3 of
          // the lane, or every a.
          const float inv0 = __uint_as_float((254u - (mine & 0xFFu)) << 23);  // 2^-e, normal
          const float inv1 = __uint_as_float((254u - (mine >> 16)) << 23);
          const F2 i0 = f2(inv0, inv0), i1 = f2(inv1, inv1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[u].a[i] = f2_mul(v[u].a[i], kHalf || i < 2 ? i0 : i1);
            v[u].b[i] = f2_mul(v[u].b[i], !kHalf && i < 2 ? i0 : i1);
          }
          from_pairs<kHalf>(v[u], x[u], y[u]);
          if (now.real && u < left) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float(&z)[8] = c ? y[u] : x[u];
              *reinterpret_cast<uint2*>(bytes + 64 * c) = make_uint2(cvt_e4m3x4(z[0], z[1], z[2], z[3]),
                                                                     cvt_e4m3x4(z[4], z[5], z[6], z[7]));
            }
          }
          sf += heads_per_step * 512;
          bytes += heads_per_step * 128;
        }
      } else {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (now.real && u < left) {
            if (kOut == kRopeBf16) {
              chunk_store(out16, x[u]);
              chunk_store(out16 + 64, y[u]);
            } else {
              chunk_store(out32, x[u]);
              chunk_store(out32 + 64, y[u]);
            }
          }
          out16 += kOut == kRopeBf16 ? out_step : 0;
          out32 += kOut == kRopeF32 ? out_step : 0;
        }
      }
      head += kBatch * heads_per_step;
    }
  }
  cp_async_wait<0>();
}

// The backward pass of four rows (a step): d becomes dx, and acc gains the weight's gradient where `on`.
template <typename T, bool kHalf>
__device__ __forceinline__ void rope_bwd_step(const RopeParams& p, uint32_t rows, const float* cs, const Pairs& w,
                                              bool on, int lane, F2 (&acc)[8], Pairs& d) {
  const int j = lane & 7;
  const F2 minus = f2(-1.f, -1.f);
  RawRow<T> rx, rg;
  rx.load_shared(rows, lane);
  rg.load_shared(rows + rope_bwd_stage<T>() / 2, lane);
  float u[8], v[8];
  rg.get(0, u);
  rg.get(1, v);
  Pairs g = to_pairs<kHalf>(u, v);
  rx.get(0, u);
  rx.get(1, v);
  const Pairs x = to_pairs<kHalf>(u, v);
  F2 ss = f2(0.f, 0.f), hx = f2(0.f, 0.f);
  F2 gx[8];
  F2 c[4], sn[4];
  turn_pairs(cs, j, c, sn);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // Back by the angle: g_a = dy_a c + dy_b s, g_b = dy_b c - dy_a s.
    const F2 a = f2_fma(g.a[i], c[i], f2_mul(g.b[i], sn[i]));
    const F2 b = f2_fma(g.b[i], c[i], f2_mul(f2_mul(g.a[i], minus), sn[i]));
    g.a[i] = a;
    g.b[i] = b;
    gx[i] = f2_mul(a, x.a[i]);
    gx[4 + i] = f2_mul(b, x.b[i]);
    hx = f2_fma(gx[i], w.a[i], hx);
    hx = f2_fma(gx[4 + i], w.b[i], hx);
    ss = f2_fma(x.a[i], x.a[i], ss);
    ss = f2_fma(x.b[i], x.b[i], ss);
  }
  float r = 1.f, q = 0.f;  // dx = r g w + q x
  if (p.norm) {
    r = rsqrt_newton(row_sum(f2_sum(ss)) * (1.f / 128.f) + p.eps);
    q = row_sum(f2_sum(hx)) * (-1.f / 128.f) * r * r * r;
  }
  const F2 r2 = f2(r, r), q2 = f2(q, q);
  const F2 ra = on ? r2 : f2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[i] = f2_fma(gx[i], ra, acc[i]);
    acc[4 + i] = f2_fma(gx[4 + i], ra, acc[4 + i]);
    d.a[i] = f2_fma(f2_mul(g.a[i], w.a[i]), r2, f2_mul(x.a[i], q2));
    d.b[i] = f2_fma(f2_mul(g.b[i], w.b[i]), r2, f2_mul(x.b[i], q2));
  }
}

// A step's rows of x and dy (token `at`, head `head`) into a stage of the warp's ring.
template <typename T>
__device__ __forceinline__ void rope_bwd_load(const RopeTensor& t, int64_t at, int head, uint32_t stage, int lane) {
  constexpr int kLaneElems = sizeof(T) == 2 ? 8 : 4;  // elements of a copy
  const int e = kLaneElems * (lane & 7);
  row_async(stage, static_cast<const T*>(t.x) + at * t.tok_stride + head * t.head_stride + e, lane);
  row_async(stage + rope_bwd_stage<T>() / 2, static_cast<const T*>(t.dy) + at * t.dy_tok + head * t.dy_head + e, lane);
}

template <typename T, bool kHalf>
__device__ __forceinline__ void rope_bwd_store(const RopeTensor& t, int64_t at, int head, const Pairs& d, int j) {
  float u[8], v[8];
  from_pairs<kHalf>(d, u, v);
  T* dst = static_cast<T*>(t.out) + at * t.out_tok + head * t.out_head + 8 * j;
  chunk_store(dst, u);
  chunk_store(dst + 64, v);
}

__device__ __forceinline__ void clear(F2 (&acc)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = f2(0.f, 0.f);
}

// The angles of a block's next tokens, by all warps; ends with a barrier.
template <bool kHalf>
__device__ __forceinline__ void rope_bwd_angles(const RopeParams& p, const LaneTurns& turns, float (*cs)[128],
                                                int64_t tok0, int ntok) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int s = warp; s < ntok; s += kRopeWarps) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      put_turn<kHalf>(cs[s], lane + 32 * i, rope_turn(rope_position(p, (tok0 + s) * p.pos_tok + turns.axis[i]), turns.f[i]));
  }
  __syncthreads();
}

// Backward with at most one weight row for all heads (8192 tokens x 32 heads of BF16: 43.5 us with the
// sums, 1.4 times the copy time of its bytes, bound by the latency of two sums of three shuffles a row and
// the reads of the angles at 16 warps an SM; its 92 warp instructions a row are half of the issue slots). Each block walks `tile` consecutive tokens, kRopeBwdTile at a time, in items of one step (four
// rows, as in the forward pass) that go round the warps, each with the next one on the way in its
// shared-memory ring. A lane's sums for its 16 channels stay in registers to the end. No atomics: the same
// sums in the same order every time.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads, 2)
qk_norm_rope_bwd_kernel(const __grid_constant__ RopeParams p, const __grid_constant__ RopePlan plan) {
  constexpr int kStage = rope_bwd_stage<T>();
  extern __shared__ __align__(16) uint8_t rope_smem[];
  float(*cs)[128] = reinterpret_cast<float(*)[128]>(rope_smem);                               // [kRopeBwdTile]
  float(*sums)[128] = reinterpret_cast<float(*)[128]>(rope_smem + kRopeBwdTile * 128 * 4);  // [4 * kRopeWarps]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane >> 3, j = lane & 7;
  const uint32_t ring = smem_u32(sums + 4 * kRopeWarps) + warp * 2 * kStage;
  cudaTriggerProgrammaticLaunchCompletion();  // every block runs at once: the sums may be set up already
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.tile;
  const int64_t last = min(first + p.tile, p.tokens);
  float* part = p.partials + static_cast<int64_t>(blockIdx.x) * (p.w_rows[0] + p.w_rows[1]) * 128;
  const int heads_per_step = p.quad ? 4 : 1;
  const int head0 = p.quad ? grp : 0;
  const int per_place = p.quad ? 1 : 4;
  const int in_place = p.quad ? 0 : grp;
  const LaneTurns turns = lane_turns(p, plan, lane);
  bool turned = false;  // one tile of tokens: its angles serve Q and K

#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const RopeTensor& t = p.t[which];
    if (t.heads == 0) continue;
    const int steps = t.heads / heads_per_step;  // (quad: multiples of four)
    F2 acc[8];
    clear(acc);
    const Pairs w = weight_pairs<kHalf>(p, t, 0, j);
    for (int64_t tok0 = first; tok0 < last; tok0 += kRopeBwdTile) {
      const int ntok = static_cast<int>(min(static_cast<int64_t>(kRopeBwdTile), last - tok0));
      const int all = (ntok + per_place - 1) / per_place * steps;
      // This warp's items: (place, step) number warp, warp + 8, ..., steps fastest.
      int place = 0, step = warp;
      auto settle = [&]() {
        while (step >= steps) {
          step -= steps;
          ++place;
        }
      };
      settle();
      // A token that does not exist reads the last one there is and counts for nothing.
      auto load = [&](int stage) {
        rope_bwd_load<T>(t, tok0 + min(place * per_place + in_place, ntok - 1), step * heads_per_step + head0,
                         ring + stage * kStage, lane);
      };
      if (warp < all) load(0);
      cp_async_commit();
      if (!turned) {
        if (last - first > kRopeBwdTile) __syncthreads();  // the angles of the previous tokens have been read
        rope_bwd_angles<kHalf>(p, turns, cs, tok0, ntok);
        turned = last - first <= kRopeBwdTile;
      }
      int stage = 0;
#pragma unroll 1
      for (int it = warp; it < all; it += kRopeWarps, stage ^= 1) {
        const int s = place * per_place + in_place;
        const int head = step * heads_per_step + head0;
        if (sizeof(T) == 4) __syncwarp();  // the stage to fill has been read (FP32: by other lanes too)
        step += kRopeWarps;
        settle();
        if (it + kRopeWarps < all) load(stage ^ 1);
        cp_async_commit();
        cp_async_wait<1>();
        if (sizeof(T) == 4) __syncwarp();
        Pairs d;
        rope_bwd_step<T, kHalf>(p, ring + stage * kStage, cs[min(s, ntok - 1)], w, s < ntok, lane, acc, d);
        if (s < ntok) rope_bwd_store<T, kHalf>(t, tok0 + s, head, d, j);
      }
      cp_async_wait<0>();
      __syncwarp();
    }
    if (p.w_rows[which] == 1) {
      __syncthreads();
      Pairs v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v.a[i] = acc[i];
        v.b[i] = acc[4 + i];
      }
      float x[8], y[8];
      from_pairs<kHalf>(v, x, y);
      chunk_store(&sums[warp * 4 + grp][8 * j], x);
      chunk_store(&sums[warp * 4 + grp][64 + 8 * j], y);
      __syncthreads();
      if (threadIdx.x < 128) {
        float sum = 0.f;
#pragma unroll 8
        for (int k = 0; k < 4 * kRopeWarps; ++k) sum += sums[k][threadIdx.x];
        part[which * p.w_rows[0] * 128 + threadIdx.x] = sum;
      }
    }
  }
}

// Backward with a weight row per head. A warp keeps a step (four heads, or one) while it walks the block's
// tokens, so that a head's sums are complete in its lanes and go straight to the block's row of partials.
// The steps left when the others have gone round the eight warps evenly are split: a warp takes a
// part of the tokens, and the parts meet in shared memory (2,740 tokens x 40 FP32 heads: two of the ten
// steps, in four parts each; 37.9 us with the sums, where a block that took one step at a time
// over all its warps, with a barrier after each, took 47.9).
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads, 2)
qk_norm_rope_bwd_heads_kernel(const __grid_constant__ RopeParams p, const __grid_constant__ RopePlan plan) {
  constexpr int kStage = rope_bwd_stage<T>();
  extern __shared__ __align__(16) uint8_t rope_smem[];
  float(*cs)[128] = reinterpret_cast<float(*)[128]>(rope_smem);  // [kRopeBwdTile]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane >> 3, j = lane & 7;
  float(*sums)[128] = reinterpret_cast<float(*)[128]>(rope_smem + kRopeBwdTile * 128 * 4);  // [4 * kRopeWarps]
  const uint32_t ring = smem_u32(sums + 4 * kRopeWarps) + warp * 2 * kStage;
  cudaTriggerProgrammaticLaunchCompletion();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.tile;
  const int64_t last = min(first + p.tile, p.tokens);
  const int part_rows = p.w_rows[0] + p.w_rows[1];
  const int heads_per_step = p.quad ? 4 : 1;
  const int head0 = p.quad ? grp : 0;
  const int per_place = p.quad ? 1 : 4;
  const int in_place = p.quad ? 0 : grp;
  const int steps_q = p.t[0].heads / heads_per_step;
  const int steps = steps_q + p.t[1].heads / heads_per_step;
  const int whole = steps / kRopeWarps * kRopeWarps;  // steps that go round the warps evenly
  const int rest = steps - whole;
  const int splits = rest ? kRopeWarps / rest : 1;  // parts of each of the others: at most one a warp
  const int units = whole + rest * splits;
  float* part = p.partials + static_cast<int64_t>(blockIdx.x) * part_rows * 128;
  const LaneTurns turns = lane_turns(p, plan, lane);

#pragma unroll 1
  for (int64_t tok0 = first; tok0 < last; tok0 += kRopeBwdTile) {
    const int ntok = static_cast<int>(min(static_cast<int64_t>(kRopeBwdTile), last - tok0));
    const int places = (ntok + per_place - 1) / per_place;
    if (tok0 != first) __syncthreads();  // the angles of the previous tokens have been read
    rope_bwd_angles<kHalf>(p, turns, cs, tok0, ntok);
    // A unit's step and places; a part may have none.
    auto enter = [&](int unit, int& step, int& place, int& end) {
      step = unit < whole ? unit : whole + (unit - whole) / splits;
      const int i = unit < whole ? 0 : (unit - whole) % splits, n = unit < whole ? 1 : splits;
      place = places * i / n;
      end = places * (i + 1) / n;
    };
    // The rows to load next: the places of one unit after another.
    int rd_unit = warp, rd_step = 0, rd_place = 0, rd_end = 0;
    auto rd_enter = [&]() {
      for (; rd_unit < units; rd_unit += kRopeWarps) {
        enter(rd_unit, rd_step, rd_place, rd_end);
        if (rd_place < rd_end) break;
      }
    };
    auto load = [&](int stage) {
      if (rd_unit < units) {
        const int step = rd_step;
        const bool is_k = step >= steps_q;
        rope_bwd_load<T>(p.t[is_k], tok0 + min(rd_place * per_place + in_place, ntok - 1),
                         (is_k ? step - steps_q : step) * heads_per_step + head0, ring + stage * kStage, lane);
        if (++rd_place == rd_end) {
          rd_unit += kRopeWarps;
          rd_enter();
        }
      }
      cp_async_commit();
    };
    rd_enter();
    load(0);
    int stage = 0;
#pragma unroll 1
    for (int unit = warp; unit < units; unit += kRopeWarps) {
      int step, place, end;
      enter(unit, step, place, end);
      const bool is_k = step >= steps_q;
      const RopeTensor& t = p.t[is_k];
      const int head = (is_k ? step - steps_q : step) * heads_per_step + head0;
      const Pairs w = weight_pairs<kHalf>(p, t, head, j);
      F2 acc[8];
      clear(acc);
#pragma unroll 1
      for (; place < end; ++place, stage ^= 1) {
        const int s = place * per_place + in_place;
        if (sizeof(T) == 4) __syncwarp();  // the stage to fill has been read (FP32: by other lanes too)
        load(stage ^ 1);
        cp_async_wait<1>();
        if (sizeof(T) == 4) __syncwarp();
        Pairs d;
        rope_bwd_step<T, kHalf>(p, ring + stage * kStage, cs[min(s, ntok - 1)], w, s < ntok, lane, acc, d);
        if (s < ntok) rope_bwd_store<T, kHalf>(t, tok0 + s, head, d, j);
      }
      if (!p.quad) {  // the four tokens of a step are one head's
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[i].x += __shfl_xor_sync(0xFFFFFFFFu, acc[i].x, 8);
          acc[i].y += __shfl_xor_sync(0xFFFFFFFFu, acc[i].y, 8);
          acc[i].x += __shfl_xor_sync(0xFFFFFFFFu, acc[i].x, 16);
          acc[i].y += __shfl_xor_sync(0xFFFFFFFFu, acc[i].y, 16);
        }
      }
      if (p.quad || grp == 0) {
        const bool split = unit >= whole && splits > 1;
        float* to = (split ? sums[4 * warp + grp] : part + ((is_k ? p.w_rows[0] : 0) + head) * 128) + 8 * j;
        Pairs v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v.a[i] = acc[i];
          v.b[i] = acc[4 + i];
        }
        float x[8], y[8];
        from_pairs<kHalf>(v, x, y);
        if (tok0 != first && !split) {  // the same lanes' sums of the tokens before
          RawRow<float> before;
          before.load(to);
          float bx[8], by[8];
          before.get(0, bx);
          before.get(1, by);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] += bx[i];
            y[i] += by[i];
          }
        }
        chunk_store(to, x);
        chunk_store(to + 64, y);
      }
    }
    cp_async_wait<0>();
    __syncwarp();
    if (splits > 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < rest * heads_per_step * 128; i += kRopeThreads) {
        const int ch = i & 127, h = (i >> 7) % heads_per_step, r = (i >> 7) / heads_per_step;
        float sum = 0.f;
        for (int k = 0; k < splits; ++k) sum += sums[4 * (r * splits + k) + h][ch];
        float* to = part + ((whole + r) * heads_per_step + h) * 128 + ch;  // (the rows of Q, then those of K)
        *to = tok0 == first ? sum : *to + sum;
      }
    }
  }
}

// Sums the blocks' partial weight gradients. Grid (rows, 4): 32 channels of a row of the result for
// a block of 32 x 32 threads, so that a thread has few loads to wait for and all at once (5 us, where two
// blocks with 74 loads a thread took 10).
__global__ void __launch_bounds__(1024)
qk_norm_rope_dw_kernel(const float* partials, int blocks, int rows, int rows_q, float* dwq, float* dwk) {
  __shared__ float sums[32][33];
  cudaGridDependencySynchronize();  // launched while the backward kernel ends
  const int row = blockIdx.x, lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int ch = blockIdx.y * 32 + lane;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < (kRopeBwdBlocks + 31) / 32; ++i) {
    const int b = grp + 32 * i;
    if (b < blocks) s += __ldcg(partials + (static_cast<int64_t>(b) * rows + row) * 128 + ch);
  }
  sums[grp][lane] = s;
  __syncthreads();
  // Warp g sums channel g of the 32 over the groups.
  s = sums[lane][grp];
#pragma unroll
  for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
  if (lane == 0) (row < rows_q ? dwq + row * 128 : dwk + (row - rows_q) * 128)[blockIdx.y * 32 + grp] = s;
}

}  // namespace lpfa
