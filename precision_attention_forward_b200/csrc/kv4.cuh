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
// Both kernels stream; HBM bounds them. A row of 128 is 16 lanes: lane m holds bytes 4m..4m+3, i.e.
// two runs of four elements in two scale blocks. Page entries are looked up once per token and
// block of threads; one outside the table or the pool skips its token and records
// LPFA_ERR_INVALID_ARG in the device status word.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "quantize.cuh"

namespace lpfa {

constexpr int kKv4Threads = 256;
constexpr int kKv4Tile = 16;  // tokens of a writing block (at most)
constexpr int kKv4Batch = 4;  // rows that a half warp has in flight

// Sites of the status word for entries out of range.
enum Kv4Site : int { kKv4WriteSite = 300, kKv4ReadSite = 301, kKv4AttnLenSite = 302, kKv4AttnPageSite = 303 };

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

// Two floats -> two E2M1 codes (round to nearest even, saturate to +-6); lo in bits 0..3.
__device__ __forceinline__ uint32_t cvt_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// E8M0 exponent for E2M1 (6 = 1.5 * 2^2) of a non-negative float block maximum.
__device__ __forceinline__ int e8m0_exponent_e2m1(float amax, int floor_mode) {
  const uint32_t bits = __float_as_uint(amax);
  const int biased = static_cast<int>(bits >> 23);
  if (biased == 0) return -127;  // zero or subnormal: below 2^-126, clamps to -127
  const int e = biased - 129 + (!floor_mode && (bits & 0x7FFFFFu) > 0x400000u);
  return max(-127, min(127, e));
}

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

template <typename T>
__device__ __forceinline__ void kv4_load4(const T* p, float (&v)[4]);
template <>
__device__ __forceinline__ void kv4_load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  v[0] = __uint_as_float(u.x << 16);
  v[1] = __uint_as_float(u.x & 0xFFFF0000u);
  v[2] = __uint_as_float(u.y << 16);
  v[3] = __uint_as_float(u.y & 0xFFFF0000u);
}
template <>
__device__ __forceinline__ void kv4_load4<float>(const float* p, float (&v)[4]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}

// Grid (token tiles, 2): K for y = 0, V for y = 1. Rows are taken token by token within a head, so
// that the 64-byte rows that neighbouring half warps write are neighbours in the page.
template <typename T>
__global__ void __launch_bounds__(kKv4Threads) kv4_write_kernel(const __grid_constant__ Kv4WriteParams p) {
  __shared__ int64_t slot_of[kKv4Tile];
  const int lane = threadIdx.x & 31, l16 = lane & 15, hw = threadIdx.x >> 4;
  const int tok0 = blockIdx.x * p.tile;
  const int ntok = min(p.tile, p.tokens - tok0);
  const int y = blockIdx.y;
  if (threadIdx.x < ntok) {
    const int tok = tok0 + threadIdx.x;
    const int seq = find_seq(p.cu_seqlens, p.num_seqs, tok);
    const int64_t at = static_cast<int64_t>(tok) - __ldg(p.cu_seqlens + seq) + (p.start ? __ldg(p.start + seq) : 0);
    const bool ok = !p.start || __ldg(p.start + seq) >= 0;
    slot_of[threadIdx.x] = kv4_slot(p.c, seq, ok ? at : -1, kKv4WriteSite);
  }
  __syncthreads();
  const T* x = static_cast<const T*>(p.x[y]);
  const int g = l16 >> 1;        // run of four elements within a block
  const int b0 = (l16 & 1) * 2;  // this lane's two blocks: b0, b0 + 1
  const int rows = ntok * p.c.heads;
  const float per_tok = 1.f / static_cast<float>(ntok);
  constexpr int kHalves = kKv4Threads / 16;
#pragma unroll 1
  for (int base = hw & ~1; base < rows; base += kHalves * kKv4Batch) {
    float v[kKv4Batch][2][4];
    int64_t row[kKv4Batch];
#pragma unroll
    for (int u = 0; u < kKv4Batch; ++u) {
      const int r = base + kHalves * u + (hw & 1);
      row[u] = -1;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i >> 2][i & 3] = 0.f;
      if (r < rows) {
        const int head = static_cast<int>((static_cast<float>(r) + 0.5f) * per_tok);  // r / ntok, r < 2^16
        const int s = r - head * ntok;
        if (slot_of[s] >= 0) {
          row[u] = kv4_row(p.c, slot_of[s], head);
          const T* src = x + (tok0 + s) * p.tok_stride[y] + head * p.head_stride[y] + 32 * b0 + 4 * g;
          kv4_load4<T>(src, v[u][0]);
          kv4_load4<T>(src + 32, v[u][1]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kKv4Batch; ++u) {
      uint32_t codes = 0, sf = 0;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float amax = fmaxf(fmaxf(fabsf(v[u][b][0]), fabsf(v[u][b][1])), fmaxf(fabsf(v[u][b][2]), fabsf(v[u][b][3])));
#pragma unroll
        for (int m = 8; m > 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, m));
        const int e = e8m0_exponent_e2m1(amax, p.floor_mode);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, normal
        codes |= (cvt_e2m1x2(v[u][b][0] * inv, v[u][b][1] * inv) |
                  (cvt_e2m1x2(v[u][b][2] * inv, v[u][b][3] * inv) << 8)) << (16 * b);
        sf |= static_cast<uint32_t>(e + 127) << (8 * b);
      }
      if (row[u] >= 0) {
        *reinterpret_cast<uint32_t*>(p.c.payload[y] + row[u] * 64 + l16 * 4) = codes;
        if (l16 < 2) *reinterpret_cast<uint16_t*>(p.c.scales[y] + row[u] * 4 + l16 * 2) = static_cast<uint16_t>(sf);
      }
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

// Grid (16 x padded 128-token blocks, 2): 8 of the 128 rows of a block, rows r0 and r0 + 1 of each
// 32-row quarter, whose scale words fill whole sectors of the atoms.
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const __grid_constant__ Kv4ReadParams p) {
  __shared__ int64_t slot_of[8];
  __shared__ int tok_of[8];  // -1: a padding row
  extern __shared__ __align__(16) uint32_t kv4_sf[];  // [head][8]
  const int lane = threadIdx.x & 31, l16 = lane & 15, hw = threadIdx.x >> 4;
  const int block = blockIdx.x >> 4, r0 = (blockIdx.x & 15) * 2;
  const int y = blockIdx.y;
  if (threadIdx.x < 8) {
    const int seq = find_seq(p.scale_off, p.num_seqs, block);
    const int first = __ldg(p.cu_seqlens + seq);
    const int in_seq = (block - __ldg(p.scale_off + seq)) * 128 + r0 + (threadIdx.x & 1) + 32 * (threadIdx.x >> 1);
    const bool real = in_seq < __ldg(p.cu_seqlens + seq + 1) - first;
    const int start = p.start ? __ldg(p.start + seq) : 0;
    tok_of[threadIdx.x] = real ? first + in_seq : -1;
    slot_of[threadIdx.x] =
        real ? kv4_slot(p.c, seq, start >= 0 ? static_cast<int64_t>(start) + in_seq : -1, kKv4ReadSite) : -1;
  }
  __syncthreads();
  const int g = l16 >> 1, b0 = (l16 & 1) * 2;
  const int rows = 8 * p.c.heads;
  constexpr int kHalves = kKv4Threads / 16;
#pragma unroll 1
  for (int base = hw; base < rows; base += kHalves * kKv4Batch) {
    uint32_t codes[kKv4Batch], sf[kKv4Batch];
#pragma unroll
    for (int u = 0; u < kKv4Batch; ++u) {
      const int r = base + kHalves * u;
      codes[u] = 0;
      sf[u] = 0x7F7F7F7Fu;
      if (r < rows && slot_of[r & 7] >= 0) {
        const int64_t row = kv4_row(p.c, slot_of[r & 7], r >> 3);
        codes[u] = *reinterpret_cast<const uint32_t*>(p.c.payload[y] + row * 64 + l16 * 4);
        if (l16 == 0) sf[u] = *reinterpret_cast<const uint32_t*>(p.c.scales[y] + row * 4);
      }
    }
#pragma unroll
    for (int u = 0; u < kKv4Batch; ++u) {
      const int r = base + kHalves * u;
      if (r >= rows) break;
      const int s = r & 7, head = r >> 3;
      if (tok_of[s] >= 0) {
        uint8_t* dst = p.payload[y] + (static_cast<int64_t>(tok_of[s]) * p.c.heads + head) * 128 + 32 * b0 + 4 * g;
        *reinterpret_cast<uint32_t*>(dst) = e2m1x4_to_e4m3x4(codes[u] & 0xFFFFu);
        *reinterpret_cast<uint32_t*>(dst + 32) = e2m1x4_to_e4m3x4(codes[u] >> 16);
      }
      if (l16 == 0) kv4_sf[head * 8 + (s & 1) * 4 + (s >> 1)] = sf[u];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.c.heads; i += kKv4Threads) {
    const int row = i & 1, head = i >> 1;
    *reinterpret_cast<uint4*>(p.scales[y] + (static_cast<int64_t>(block) * p.c.heads + head) * 512 + (r0 + row) * 16) =
        *reinterpret_cast<const uint4*>(kv4_sf + head * 8 + row * 4);
  }
}

}  // namespace lpfa
