// kv4.cuh -- a paged key/value cache in MXFP4: writing new tokens into it and reading them back as
// MXFP8 tensors.
//
// Format: E2M1 codes (values 0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives) with one E8M0 power of
// two 2^e per 32 elements along head_dim. e is the smallest with amax <= 6 * 2^e (RCEIL) or
// floor(log2 amax) - 2 (FLOOR), clamped to [-127, 127], and -127 for amax 0; the code is
// E2M1(x * 2^-e), one round to nearest even, saturating. 17/32 byte per element.
//
// Layout: payload (pages, heads, page_size, 64) and scales (pages, heads, page_size, 4) for each of
// K and V. Element 32 b + 4 g + 2 j + n of a row is the low (n = 0) or high (n = 1) nibble of byte
// 8 g + 2 b + j: the order in which the attention's matrix fragments take a row, so that a lane's
// share of it is one 16-byte (K) or 8-byte (V) load and every fragment lies within one scale block.
// Token p of sequence s is row p % page_size of page table[s][p / page_size].
//
// E2M1 is a subset of E4M3 and the scale rule's power of two is the same kind of byte, so reading a
// cached row back as MXFP8 is exact: codes are looked up, scales are copied.
//
// Both kernels stream; HBM bounds them. Four lanes own a row: lane t holds the row's 16 bytes 16 t ..
// 16 t + 15, which are the elements 8 t .. 8 t + 7 of each of the four scale blocks, so a lane reads
// (or writes) whole 16-byte (8-byte) runs, a block's maximum is two shuffles, and a warp moves eight
// rows at a time. (With 16 lanes to a row, four bytes each, the same work took 81 and 49 warp
// instructions a row for writing and reading and reached a third of the copy bandwidth.) Page entries
// are looked up once per token and block of threads; one outside the table or the pool skips its token
// and records LPFA_ERR_INVALID_ARG in the device status word.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "qk_norm_rope.cuh"
#include "quantize.cuh"

namespace lpfa {

constexpr int kKv4Threads = 256;
constexpr int kKv4Tile = 32;  // tokens of a block, at most
constexpr int kKv4Rows = kKv4Threads / 4;  // rows that a block has in hand at a time

// Sites of the status word for entries out of range.
enum Kv4Site : int { kKv4WriteSite = 300, kKv4ReadSite = 301, kKv4AttnLenSite = 302, kKv4AttnPageSite = 303,
                    kKv4AttnWaitSite = 304 /* a bounded wait ran out */ };

struct Kv4Cache {
  uint8_t* payload[2];  // K, V
  uint8_t* scales[2];
  int pages, heads, page_size, page_shift;
  const int32_t* table;  // (sequences, width), row stride in elements
  int64_t table_stride;
  int width;
};

__device__ __forceinline__ void kv4_bad_entry(int site) {
  if (atomicCAS(&g_lpfa_status[0], 0, 1 /* LPFA_ERR_INVALID_ARG */) == 0) atomicExch(&g_lpfa_status[1], site);
}

// Row (page * page_size + row in page) of token `at` of sequence `seq`, or -1. The row of head h is
// then at ((page * heads + h) * page_size + row): see kv4_row.
__device__ __forceinline__ int64_t kv4_slot(const Kv4Cache& c, int seq, int64_t at, int site) {
  if (at >= 0 && (at >> c.page_shift) < c.width) {
    const int page = __ldg(c.table + seq * c.table_stride + (at >> c.page_shift));
    if (page >= 0 && page < c.pages) return (static_cast<int64_t>(page) << c.page_shift) + (at & (c.page_size - 1));
  }
  kv4_bad_entry(site);
  return -1;
}

__device__ __forceinline__ int64_t kv4_row(const Kv4Cache& c, int64_t slot, int head) {
  return (((slot >> c.page_shift) * c.heads + head) << c.page_shift) + (slot & (c.page_size - 1));
}

// Four floats -> four E2M1 codes (round to nearest even, saturate to +-6), the first in bits 0..3.
__device__ __forceinline__ uint32_t cvt_e2m1x4(F2 a, F2 b) {
  uint16_t r;
  asm("{\n\t.reg .b8 lo, hi;\n\tcvt.rn.satfinite.e2m1x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 hi, %4, %3;\n\tmov.b16 %0, {lo, hi};\n\t}"
      : "=h"(r) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Scale byte for E2M1 (6 = 1.5 * 2^2) of a block maximum: e + 127 with e the smallest with
// amax <= 6 * 2^e (`up` carries a mantissa above 1.5 into the exponent) or, with up 0,
// floor(log2 amax) - 2; a zero or subnormal maximum gives 0, the clamp at 2^-127.
__device__ __forceinline__ uint32_t e2m1_scale_byte(float amax, uint32_t up) {
  return max((__float_as_uint(amax) + up) >> 23, 2u) - 2u;
}
constexpr uint32_t kE2m1Up = 0x3FFFFFu;

// Four E2M1 codes (nibbles 0..3) -> four E4M3 codes, exactly.
__device__ __forceinline__ uint32_t e2m1x4_to_e4m3x4(uint32_t nibbles) {
  // Magnitudes by a byte lookup: 0 .5 1 1.5 | 2 3 4 6 as E4M3.
  const uint32_t mag = __byte_perm(0x3C383000u, 0x4C484440u, nibbles & 0x7777u);
  const uint32_t s = nibbles & 0x8888u;
  return mag | ((s & 0x8u) << 4) | ((s & 0x80u) << 8) | ((s & 0x800u) << 12) | ((s & 0x8000u) << 16);
}

struct Kv4WriteParams {
  Kv4Cache c;
  const void* x[2];  // K, V: (T, heads, 128)
  int64_t tok_stride[2], head_stride[2];
  int num_seqs;
  const int32_t* cu_seqlens;
  const int32_t* start;  // tokens already cached per sequence, or NULL (0)
  int tokens;
  int tile;
  int floor_mode;
};

// Grid (token tiles, 2): K for y = 0, V for y = 1. Rows are taken token by token within a head: the
// 64-byte rows that neighbouring lanes write are neighbours in the page, and what they read are whole
// 256-byte (512-byte) rows.
template <typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_write_kernel(const __grid_constant__ Kv4WriteParams p) {
  __shared__ int64_t slot_of[kKv4Tile];
  const int t = threadIdx.x & 3;
  const int tok0 = blockIdx.x * p.tile;
  const int ntok = min(p.tile, p.tokens - tok0);
  const int y = blockIdx.y;
  if (threadIdx.x < ntok) {
    const int tok = tok0 + threadIdx.x;
    const int seq = find_seq(p.cu_seqlens, p.num_seqs, tok);
    const int start = p.start ? __ldg(p.start + seq) : 0;
    const int64_t at = static_cast<int64_t>(tok) - __ldg(p.cu_seqlens + seq) + start;
    slot_of[threadIdx.x] = kv4_slot(p.c, seq, start >= 0 ? at : -1, kKv4WriteSite);
  }
  __syncthreads();
  const T* x = static_cast<const T*>(p.x[y]) + tok0 * p.tok_stride[y] + 8 * t;
  const int rows = ntok * p.c.heads;
  const float per_tok = 1.f / static_cast<float>(ntok);
  const uint32_t up = p.floor_mode ? 0u : kE2m1Up;
#pragma unroll 1
  for (int base = (threadIdx.x >> 5) * 8; base < rows; base += kKv4Rows) {  // the same for the whole warp
    const int r = base + ((threadIdx.x & 31) >> 2);
    const int head = static_cast<int>((static_cast<float>(r) + 0.5f) * per_tok);  // r / ntok, r < 2^16
    const int s = r - head * ntok;
    const int64_t slot = r < rows ? slot_of[s] : -1;
    uint4 raw[sizeof(T)][2];  // BF16: [0..1][0..1] are blocks 0..3; FP32: [block][half]
    const uint4* src = reinterpret_cast<const uint4*>(x + s * p.tok_stride[y] + head * p.head_stride[y]);
#pragma unroll
    for (int i = 0; i < 2 * static_cast<int>(sizeof(T)); ++i) {
      raw[i >> 1][i & 1] = make_uint4(0, 0, 0, 0);
      if (slot >= 0) raw[i >> 1][i & 1] = __ldg(src + (sizeof(T) == 2 ? 4 * i : 8 * (i >> 1) + (i & 1)));
    }
    uint32_t h[2][4];  // the four runs of two bytes: [run 2t or 2t + 1][block]
    uint32_t sf = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float v[8];
      if (sizeof(T) == 2) {
        const uint4 u = raw[b >> 1][b & 1];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      } else {
        const uint4 lo = raw[b % sizeof(T)][0], hi = raw[b % sizeof(T)][1];
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
      }
      float amax = chunk_amax(v);
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      const uint32_t byte = e2m1_scale_byte(amax, up);
      const float inv = __uint_as_float((254u - byte) << 23);  // 2^-e, normal
      const F2 inv2 = f2(inv, inv);
      F2 q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = f2_mul(f2(v[2 * i], v[2 * i + 1]), inv2);
      h[0][b] = cvt_e2m1x4(q[0], q[1]);
      h[1][b] = cvt_e2m1x4(q[2], q[3]);
      sf |= byte << (8 * b);
    }
    if (slot >= 0) {
      const int64_t row = kv4_row(p.c, slot, head);
      *reinterpret_cast<uint4*>(p.c.payload[y] + row * 64 + t * 16) =
          make_uint4(h[0][0] | (h[0][1] << 16), h[0][2] | (h[0][3] << 16), h[1][0] | (h[1][1] << 16),
                     h[1][2] | (h[1][3] << 16));
      if (t == 0) *reinterpret_cast<uint32_t*>(p.c.scales[y] + row * 4) = sf;
    }
  }
}

struct Kv4ReadParams {
  Kv4Cache c;
  uint8_t* payload[2];  // (T, heads, 128) E4M3
  uint8_t* scales[2];   // atoms
  int num_seqs;
  const int32_t* cu_seqlens;
  const int32_t* scale_off;
  const int32_t* start;
};

// Grid (4 x padded 128-token blocks, 2): 32 of the 128 rows of a block, rows r0 .. r0 + 7 of each
// 32-row quarter, whose scale words fill whole sectors of the atoms.
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const __grid_constant__ Kv4ReadParams p) {
  __shared__ int64_t slot_of[kKv4Tile];
  __shared__ int tok_of[kKv4Tile];  // -1: a padding row
  extern __shared__ __align__(16) uint32_t kv4_sf[];  // [head][row of the quarter][quarter]
  const int t = threadIdx.x & 3;
  const int block = blockIdx.x >> 2, r0 = (blockIdx.x & 3) * 8;
  const int y = blockIdx.y;
  if (threadIdx.x < kKv4Tile) {
    const int seq = find_seq(p.scale_off, p.num_seqs, block);
    const int first = __ldg(p.cu_seqlens + seq);
    const int in_seq = (block - __ldg(p.scale_off + seq)) * 128 + r0 + (threadIdx.x & 7) + 32 * (threadIdx.x >> 3);
    const bool real = in_seq < __ldg(p.cu_seqlens + seq + 1) - first;
    const int start = p.start ? __ldg(p.start + seq) : 0;
    tok_of[threadIdx.x] = real ? first + in_seq : -1;
    slot_of[threadIdx.x] =
        real ? kv4_slot(p.c, seq, start >= 0 ? static_cast<int64_t>(start) + in_seq : -1, kKv4ReadSite) : -1;
  }
  __syncthreads();
  const int rows = kKv4Tile * p.c.heads;
#pragma unroll 2
  for (int r = threadIdx.x >> 2; r < rows; r += kKv4Rows) {
    const int s = r & (kKv4Tile - 1), head = r / kKv4Tile;
    const int64_t slot = slot_of[s];
    uint4 codes = make_uint4(0, 0, 0, 0);
    uint32_t sf = 0x7F7F7F7Fu;
    if (slot >= 0) {
      const int64_t row = kv4_row(p.c, slot, head);
      codes = *reinterpret_cast<const uint4*>(p.c.payload[y] + row * 64 + t * 16);
      if (t == 0) sf = *reinterpret_cast<const uint32_t*>(p.c.scales[y] + row * 4);
    }
    if (tok_of[s] >= 0) {
      uint8_t* dst = p.payload[y] + (static_cast<int64_t>(tok_of[s]) * p.c.heads + head) * 128 + 8 * t;
      const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t both = __byte_perm(w[b >> 1], w[2 + (b >> 1)], (b & 1) ? 0x7632 : 0x5410);
        *reinterpret_cast<uint2*>(dst + 32 * b) =
            make_uint2(e2m1x4_to_e4m3x4(both & 0xFFFFu), e2m1x4_to_e4m3x4(both >> 16));
      }
    }
    if (t == 0) kv4_sf[head * kKv4Tile + (s & 7) * 4 + (s >> 3)] = sf;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * p.c.heads; i += kKv4Threads) {
    const int row = i & 7, head = i >> 3;
    *reinterpret_cast<uint4*>(p.scales[y] + (static_cast<int64_t>(block) * p.c.heads + head) * 512 + (r0 + row) * 16) =
        *reinterpret_cast<const uint4*>(kv4_sf + head * kKv4Tile + row * 4);
  }
}

}  // namespace lpfa
