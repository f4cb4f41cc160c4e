// attn_kv4.cuh -- attention of a few query tokens per sequence over the paged MXFP4 cache (kv4.cuh).
//
// For query row q (one token and query head) of a sequence with n cached tokens, over the keys it
// may see (all n, or with `causal` those up to its own token, the last of the cached ones being the
// last query token's):
//   s_j = q . k_j / sqrt(128),  O = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),
//   LSE = m + log sum_j e^(s_j - m).  No key: O = 0, LSE = -inf.
//
// What bounds it: the cache is read once, 136 bytes per key and head for K and V, and each byte feeds
// 4 flops per query row, so HBM for up to 16 rows; next to it the conversion from 4 bits (one
// instruction for two elements, and one more to transpose V's), which has to hide behind the loads.
// Why mma.sync and not tcgen05: a query tile has 8 or 16 rows, a sixteenth of the tensor-memory
// accumulator's 128, and converted operands would have to pass through shared memory; in registers
// the codes go from the load through cvt straight into the fragment.
//
// Mapping. Keys are the M = 16 dimension of m16n8k16, queries the N = 8 dimension, so one query
// costs no more than eight. S^T = K Q^T: a lane's 16-byte share of a key row is its part of all eight
// fragments, and each fragment lies within one 32-element scale block, so the E8M0 scale multiplies
// an FP32 partial sum (4 per key and query) instead of every element, exactly for every scale. Q is
// scaled per row by a power of two into FP16's range, which holds a BF16 value exactly down to
// 2^-29 of the row's largest. O^T = V^T P^T: the fragment's channels lie in one scale block too, so
// V's scale multiplies P (8 half2 products per 16 keys) and V's codes stay unscaled.
// P is FP16 with the bias 2^8 and V's scale relative to the warp's largest one with the bias 2^7:
// both keep 11 bits over 2^-22 of the largest and vanish only below 2^-29, and the product stays
// under 2^15. S, the softmax statistics and O are FP32.
//
// Split. A block has four warps, each walking its own tiles of 32 keys with its own running maximum
// and accumulators (no barrier in the loop); cp.async keeps kAttn4Stages tiles per warp on the way.
// The blocks of a cluster share the keys of one (sequence, key head, query tile) and join their
// partial results through distributed shared memory: one launch, no workspace, and always the same
// order of sums.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "ptx.cuh"

namespace lpfa {

constexpr int kAttn4Warps = 4;
constexpr int kAttn4Threads = 32 * kAttn4Warps;
constexpr int kAttn4Keys = 32;    // keys of a warp's tile
constexpr int kAttn4Stages = 4;   // tiles per warp in shared memory
constexpr int kAttn4StageBytes = kAttn4Keys * (64 + 64 + 4 + 4);
constexpr int kAttn4Ring = kAttn4Stages * kAttn4StageBytes;
constexpr int kAttn4MaxSplit = 8;
constexpr float kAttn4PBias = 8.f;  // P is 2^8 e^(s - m)
constexpr int kAttn4VBias = 7;      // V's scale is 2^(7 + byte - largest byte)

struct Attn4Params {
  Kv4Cache c;
  const __nv_bfloat16* q;  // (Tq, heads_q, 128), strides in elements
  int64_t q_tok, q_head;
  const int32_t* cu_q;
  const int32_t* kv_lens;
  int num_seqs, heads_q, group;  // group: query heads per key head
  int tiles;                     // query tiles of the longest sequence
  int causal;
  int splits;
  int64_t total_q;
  __nv_bfloat16* out;  // (Tq, heads_q, 128)
  float* lse;          // (heads_q, Tq)
};

// Two E2M1 codes (a byte) -> f16x2, exactly.
template <int kByte>
__device__ __forceinline__ uint32_t cvt_e2m1x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}"
      : "=r"(r) : "r"(w), "n"(kByte));
  return r;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float dsmem_ld(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(v) : "r"(addr), "r"(rank));
  return v;
}

// The largest of a word's four bytes.
__device__ __forceinline__ uint32_t max_byte(uint32_t w) {
  w = __vmaxu4(w, w >> 16);
  return max(w & 0xFFu, (w >> 8) & 0xFFu);
}

// Physical key of row m (0..7) of an 8-row half of a fragment: 0 5 1 4 2 7 3 6. With it the eight
// rows that a quarter warp reads for K, and the four that a half warp reads for V, fall into
// different banks (V's 16-byte chunks are exchanged in rows 2, 3, 6, 7 as well).
__device__ __forceinline__ int attn4_key(int m) { return (m & 1) ? 4 + ((m >> 1) ^ 1) : m >> 1; }

// kTiles: tiles of 8 query rows that a block holds (rows = query tokens x query heads of a key head).
template <int kTiles>
__global__ void __launch_bounds__(kAttn4Threads) attn_kv4_kernel(const __grid_constant__ Attn4Params p) {
  constexpr int kRows = 8 * kTiles;
  constexpr int kPitch = 132;  // floats per row of a partial O
  extern __shared__ __align__(16) uint8_t smem4[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  // Work of this cluster: (sequence, key head, query tile), tiles fastest so that those that share
  // their keys run together.
  const uint32_t split = blockIdx.x % p.splits;
  uint32_t w = blockIdx.x / p.splits;
  const int qt = w % p.tiles;
  w /= p.tiles;
  const int kvh = w % p.c.heads;
  const int seq = w / p.c.heads;
  const int q0 = __ldg(p.cu_q + seq);
  const int lq = __ldg(p.cu_q + seq + 1) - q0;
  const int rows = lq * p.group;
  const int row0 = qt * kRows;
  if (row0 >= rows) return;  // the whole cluster

  int kv = __ldg(p.kv_lens + seq);
  const int64_t room = static_cast<int64_t>(p.c.width) << p.c.page_shift;
  if (kv < 0 || kv > room) {
    if (threadIdx.x == 0) kv4_bad_entry(kKv4AttnLenSite);
    kv = kv < 0 ? 0 : static_cast<int>(room);
  }
  // Row rr of the sequence is query token rr / group, head kvh * group + rr % group.
  const int last_tok = (min(row0 + kRows, rows) - 1) / p.group;
  const int hi = p.causal ? max(0, kv - lq + 1 + last_tok) : kv;  // keys that some row sees
  const int all_tiles = (hi + kAttn4Keys - 1) / kAttn4Keys;
  const int per_split = (all_tiles + p.splits - 1) / p.splits;
  const int tile0 = min(all_tiles, static_cast<int>(split) * per_split);
  const int tile1 = min(all_tiles, tile0 + per_split);

  // Q fragments (lane: row g, elements 32 b + 8 t .. + 7) and, for the columns 2t, 2t + 1 that a
  // lane's S holds, the factor from S to log2 units and the number of keys seen.
  uint32_t qf[kTiles][4][4];
  float c2[kTiles][2];
  int lim[kTiles][2];
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
    const int rr = row0 + 8 * n + g;
    const bool on = rr < rows;
    const int tok = on ? rr / p.group : 0;
    float v[4][8];
    float amax = 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (on)
        u = __ldg(reinterpret_cast<const uint4*>(p.q + (q0 + tok) * p.q_tok +
                                                 (kvh * p.group + rr - tok * p.group) * p.q_head + 32 * b + 8 * t));
      const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[b][2 * i] = __uint_as_float(x[i] << 16);
        v[b][2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
        amax = fmaxf(amax, fmaxf(fabsf(v[b][2 * i]), fabsf(v[b][2 * i + 1])));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    // 2^up takes the row's maximum into [2^14, 2^15); up is kept where 2^up and 2^-up are normal.
    const int ex = static_cast<int>(__float_as_uint(amax) >> 23);
    const int up = (ex == 0 || ex == 255) ? 0 : min(126, 141 - ex);
    const float scale = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[n][b][i] = half2_bits(v[b][2 * i] * scale, v[b][2 * i + 1] * scale);
    const float back = __uint_as_float(static_cast<uint32_t>(127 - up) << 23) * 0.12751743f;  // log2(e) / sqrt(128)
    const int seen = on ? (p.causal ? max(0, kv - lq + 1 + tok) : kv) : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c2[n][i] = __shfl_sync(0xFFFFFFFFu, back, (2 * t + i) * 4);
      lim[n][i] = __shfl_sync(0xFFFFFFFFu, seen, (2 * t + i) * 4);
    }
  }
  int lim_min = 0x7FFFFFFF;
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rr = row0 + 8 * n + 2 * t + i;
      if (rr < rows) lim_min = min(lim_min, lim[n][i]);  // rows that do not exist need no mask
    }
  }
  lim_min = min(lim_min, __shfl_xor_sync(0xFFFFFFFFu, lim_min, 1));
  lim_min = min(lim_min, __shfl_xor_sync(0xFFFFFFFFu, lim_min, 2));

  float o[kTiles][8][4];
  float mx[kTiles][2], l[kTiles][2];
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][d][i] = 0.f;
    mx[n][0] = mx[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
  }
  uint32_t vref = 0;  // the largest V scale byte so far, in the four bytes of a word

  uint8_t* ring = smem4 + warp * kAttn4Ring;
  const uint32_t ring_u = smem_u32(ring);
  // Table entries of the two 16-key halves of a tile (pages hold 16 tokens or more); -1 beyond hi.
  const int32_t* table = p.c.table + seq * p.c.table_stride;
  auto entries = [&](int tile) {
    const int key = tile * kAttn4Keys;
    return make_int2(key < hi ? __ldg(table + (key >> p.c.page_shift)) : -1,
                     key + 16 < hi ? __ldg(table + ((key + 16) >> p.c.page_shift)) : -1);
  };
  // Tile `tile`, whose entries are `pg`, into ring stage `st`; keys at or beyond hi become zeros.
  // Returns the halves whose page is not in the pool (bits 0 and 1): their keys are not seen.
  auto load_tile = [&](int tile, int2 pg, int st) {
    const uint32_t dst = ring_u + st * kAttn4StageBytes;
    const int key0 = tile * kAttn4Keys;
    int64_t rows_at[2];
    uint32_t missing = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = key0 + 16 * h;
      const int page = h ? pg.y : pg.x;
      rows_at[h] = -1;
      if (key < hi) {
        if (page >= 0 && page < p.c.pages) {
          rows_at[h] = (((static_cast<int64_t>(page) * p.c.heads + kvh) << p.c.page_shift)) + (key & (p.c.page_size - 1));
        } else {
          missing |= 1u << h;
          if (lane == 0) kv4_bad_entry(kKv4AttnPageSite);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 8 * j + (lane >> 2), ch = lane & 3;  // row of the tile, 16-byte chunk
      const int64_t base = rows_at[j >> 1];
      const bool on = base >= 0 && key0 + r < hi;
      const int64_t off = on ? (base + (r & 15)) * 64 + ch * 16 : 0;
      const uint32_t n = on ? 16u : 0u;
      cp_async16(dst + r * 64 + ch * 16, p.c.payload[0] + off, n);
      cp_async16(dst + 2048 + r * 64 + (ch ^ (r & 2)) * 16, p.c.payload[1] + off, n);
    }
    if (lane < 16) {
      const int r = (lane & 7) * 4;  // four keys' scale words
      const int64_t base = (lane & 4) ? rows_at[1] : rows_at[0];
      const int left = hi - key0 - r;
      const bool on = base >= 0 && left > 0;
      cp_async16(dst + 4096 + lane * 16, p.c.scales[lane >> 3] + (on ? (base + (r & 15)) * 4 : 0),
                 on ? static_cast<uint32_t>(min(16, 4 * left)) : 0u);
    }
    return missing;
  };

  const int mine = tile0 + warp;  // this warp's tiles: mine, mine + 4, ...
  uint32_t bad = 0;  // two bits per stage: halves whose page is missing
#pragma unroll
  for (int st = 0; st < kAttn4Stages - 1; ++st) {
    const int tile = mine + st * kAttn4Warps;
    if (tile < tile1) bad |= load_tile(tile, entries(tile), st) << (2 * st);
    cp_async_commit();
  }
  int st = 0;
  int2 ahead = entries(mine + (kAttn4Stages - 1) * kAttn4Warps);  // loaded a tile before they are needed
  for (int tile = mine; tile < tile1; tile += kAttn4Warps) {
    cp_async_wait<kAttn4Stages - 2>();
    __syncwarp();  // every lane's copies of this tile have landed, and the stage to refill was read
    const int next = tile + (kAttn4Stages - 1) * kAttn4Warps;
    const int nst = (st + kAttn4Stages - 1) % kAttn4Stages;
    bad &= ~(3u << (2 * nst));
    if (next < tile1) bad |= load_tile(next, ahead, nst) << (2 * nst);
    ahead = entries(next + kAttn4Warps);
    cp_async_commit();

    const uint8_t* kt = ring + st * kAttn4StageBytes;
    const uint8_t* vt = kt + 2048;
    const uint32_t* ksf = reinterpret_cast<const uint32_t*>(kt + 4096);
    const uint32_t* vsf = ksf + kAttn4Keys;

    // ---- S^T (two tiles of 16 keys): c0, c1: key attn4_key(g), c2, c3: 8 more; columns 2t, 2t + 1
    float s[2][kTiles][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r0 = 16 * h + attn4_key(g);
      const uint4 k0 = *reinterpret_cast<const uint4*>(kt + r0 * 64 + t * 16);
      const uint4 k1 = *reinterpret_cast<const uint4*>(kt + (r0 + 8) * 64 + t * 16);
      const uint32_t f0 = ksf[r0], f1 = ksf[r0 + 8];
      // Byte 2 (b % 2) + j of word b / 2 (elements 8t .. + 3 of block b) or 2 + b / 2 (8t + 4 ..).
      const uint32_t kw0[4] = {k0.x, k0.y, k0.z, k0.w}, kw1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t a[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w0 = kw0[2 * e + b / 2], w1 = kw1[2 * e + b / 2];
          a[e][0] = (b & 1) ? cvt_e2m1x2_to_f16x2<2>(w0) : cvt_e2m1x2_to_f16x2<0>(w0);
          a[e][1] = (b & 1) ? cvt_e2m1x2_to_f16x2<2>(w1) : cvt_e2m1x2_to_f16x2<0>(w1);
          a[e][2] = (b & 1) ? cvt_e2m1x2_to_f16x2<3>(w0) : cvt_e2m1x2_to_f16x2<1>(w0);
          a[e][3] = (b & 1) ? cvt_e2m1x2_to_f16x2<3>(w1) : cvt_e2m1x2_to_f16x2<1>(w1);
        }
        const float x0 = __uint_as_float(((f0 >> (8 * b)) & 0xFFu) << 23);  // byte 0 (2^-127) counts as 0
        const float x1 = __uint_as_float(((f1 >> (8 * b)) & 0xFFu) << 23);
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 2; ++e)
            mma_f16(d, a[e][0], a[e][1], a[e][2], a[e][3], qf[n][b][2 * e], qf[n][b][2 * e + 1]);
          if (b == 0) {
            s[h][n][0] = d[0] * x0;
            s[h][n][1] = d[1] * x0;
            s[h][n][2] = d[2] * x1;
            s[h][n][3] = d[3] * x1;
          } else {
            s[h][n][0] = fmaf(d[0], x0, s[h][n][0]);
            s[h][n][1] = fmaf(d[1], x0, s[h][n][1]);
            s[h][n][2] = fmaf(d[2], x1, s[h][n][2]);
            s[h][n][3] = fmaf(d[3], x1, s[h][n][3]);
          }
        }
      }
    }

    // ---- log2 units, masks, running maximum
    const int key0 = tile * kAttn4Keys + attn4_key(g);
    const uint32_t gone = (bad >> (2 * st)) & 3u;
    const bool masked = gone != 0 || (tile + 1) * kAttn4Keys > lim_min;
    float top[kTiles][2];
    bool moved = false;
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float m = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = s[h][n][2 * e + i] * c2[n][i];
            if (masked && (key0 + 16 * h + 8 * e >= lim[n][i] || ((gone >> h) & 1u))) x = -INFINITY;
            s[h][n][2 * e + i] = x;
            m = fmaxf(m, x);
          }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
        top[n][i] = m;
        moved |= m > mx[n][i];
      }
    }
    // ---- V scales: the reference follows the largest byte
    const uint32_t vw = vsf[lane];
    uint32_t big = __vmaxu4(vw, vref);
    const bool grew = big != vref;
    if (__any_sync(0xFFFFFFFFu, moved || grew)) {
      big = max_byte(big);
      big = __reduce_max_sync(0xFFFFFFFFu, big);
      const int down = static_cast<int>(vref & 0xFFu) - static_cast<int>(big);
      vref = big * 0x01010101u;
      const float fv = down < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + down) << 23);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float m = fmaxf(mx[n][i], top[n][i]);
          const float f = mx[n][i] == -INFINITY ? 0.f : ex2_approx(mx[n][i] - m);  // no key yet: o and l are 0
          mx[n][i] = m;
          l[n][i] *= f;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            o[n][d][i] *= f * fv;
            o[n][d][2 + i] *= f * fv;
          }
        }
      }
    }
    // ---- P^T as the B operand: 2^8 e^(s - m), keys 2t, 2t + 1 (and 8 more) of column g
    uint32_t pb[2][kTiles][2];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      // (no key seen so far: m = -inf, and every s of the column is -inf too)
      const float r0 = mx[n][0] == -INFINITY ? 0.f : kAttn4PBias - mx[n][0];
      const float r1 = mx[n][1] == -INFINITY ? 0.f : kAttn4PBias - mx[n][1];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float e0 = ex2_approx(s[h][n][0] + r0), e1 = ex2_approx(s[h][n][1] + r1);
        const float e2 = ex2_approx(s[h][n][2] + r0), e3 = ex2_approx(s[h][n][3] + r1);
        l[n][0] += e0 + e2;
        l[n][1] += e1 + e3;
        pb[h][n][0] = movmatrix(half2_bits(e0, e1));
        pb[h][n][1] = movmatrix(half2_bits(e2, e3));
      }
    }
    // ---- O^T += V^T P^T
    const uint32_t bias = (0x0000FFFFu & static_cast<uint32_t>(15 + kAttn4VBias - static_cast<int>(vref & 0xFFu))) * 0x00010001u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // Physical keys of fragment keys 2t, 2t + 1, 2t + 8, 2t + 9.
      const int ra = 16 * h + t, rb = 16 * h + 4 + (t ^ 1);
      const int ga = ((g >> 1) ^ (ra & 2)) * 16 + (g & 1) * 8, gb = ((g >> 1) ^ (rb & 2)) * 16 + (g & 1) * 8;
      const uint2 va = *reinterpret_cast<const uint2*>(vt + ra * 64 + ga);
      const uint2 vb = *reinterpret_cast<const uint2*>(vt + rb * 64 + gb);
      const uint2 vc = *reinterpret_cast<const uint2*>(vt + (ra + 8) * 64 + ga);
      const uint2 vd = *reinterpret_cast<const uint2*>(vt + (rb + 8) * 64 + gb);
      const uint32_t sa = vsf[ra], sb = vsf[rb], sc = vsf[ra + 8], sd = vsf[rb + 8];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        // f16 2^(7 + byte - vref) of the key pairs: exponent field, 0 (value 0) where it would be < 1.
        const uint32_t pick = 0x400u + 0x101u * static_cast<uint32_t>(b);  // byte b of the first, byte b of the second
        const uint32_t fab = __viaddmax_s16x2_relu(__byte_perm(sa, sb, pick) & 0x00FF00FFu, bias, 0u) << 10;
        const uint32_t fcd = __viaddmax_s16x2_relu(__byte_perm(sc, sd, pick) & 0x00FF00FFu, bias, 0u) << 10;
        uint32_t p0[kTiles], p1[kTiles];
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          p0[n] = half2_mul(pb[h][n][0], fab);
          p1[n] = half2_mul(pb[h][n][1], fcd);
        }
        const uint32_t wa = b < 2 ? va.x : va.y, wb = b < 2 ? vb.x : vb.y;
        const uint32_t wc = b < 2 ? vc.x : vc.y, wd = b < 2 ? vd.x : vd.y;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t xa, xb, xc, xd;
          if ((b & 1) == 0 && j == 0) {
            xa = cvt_e2m1x2_to_f16x2<0>(wa); xb = cvt_e2m1x2_to_f16x2<0>(wb);
            xc = cvt_e2m1x2_to_f16x2<0>(wc); xd = cvt_e2m1x2_to_f16x2<0>(wd);
          } else if ((b & 1) == 0) {
            xa = cvt_e2m1x2_to_f16x2<1>(wa); xb = cvt_e2m1x2_to_f16x2<1>(wb);
            xc = cvt_e2m1x2_to_f16x2<1>(wc); xd = cvt_e2m1x2_to_f16x2<1>(wd);
          } else if (j == 0) {
            xa = cvt_e2m1x2_to_f16x2<2>(wa); xb = cvt_e2m1x2_to_f16x2<2>(wb);
            xc = cvt_e2m1x2_to_f16x2<2>(wc); xd = cvt_e2m1x2_to_f16x2<2>(wd);
          } else {
            xa = cvt_e2m1x2_to_f16x2<3>(wa); xb = cvt_e2m1x2_to_f16x2<3>(wb);
            xc = cvt_e2m1x2_to_f16x2<3>(wc); xd = cvt_e2m1x2_to_f16x2<3>(wd);
          }
          const uint32_t a0 = __byte_perm(xa, xb, 0x5410), a1 = __byte_perm(xa, xb, 0x7632);
          const uint32_t a2 = __byte_perm(xc, xd, 0x5410), a3 = __byte_perm(xc, xd, 0x7632);
#pragma unroll
          for (int n = 0; n < kTiles; ++n) mma_f16(o[n][2 * b + j], a0, a1, a2, a3, p0[n], p1[n]);
        }
      }
    }
    st = st + 1 == kAttn4Stages ? 0 : st + 1;
  }
  cp_async_wait<0>();
  __syncwarp();

  // ---- join: the warp's partial (O without its bias, m, l) over its own ring, then the block's, then
  // the cluster's.
  float* part = reinterpret_cast<float*>(ring);  // [kRows][kPitch], then m[kRows], l[kRows]
  const int undo = static_cast<int>(vref & 0xFFu) - 127 - kAttn4VBias;
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 4);
      l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 8);
      l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 16);
      const int row = 8 * n + 2 * t + i;
      if (g == 0) {
        part[kRows * kPitch + row] = mx[n][i];
        part[kRows * kPitch + kRows + row] = l[n][i];
      }
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        float* to = part + row * kPitch + 32 * (d >> 1) + 4 * g + 2 * (d & 1);
        to[0] = scalbnf(o[n][d][i], undo);
        to[1] = scalbnf(o[n][d][2 + i], undo);
      }
    }
  }
  __syncthreads();
  constexpr int kRingFloats = kAttn4Ring / 4;
  const float* parts = reinterpret_cast<const float*>(smem4);
  float* joined = reinterpret_cast<float*>(smem4 + kAttn4Warps * kAttn4Ring);  // like a warp's partial
  for (int row = 0; row < kRows; ++row) {
    const int ch = threadIdx.x;
    float m = -INFINITY, lsum = 0.f, acc = 0.f;
#pragma unroll
    for (int x = 0; x < kAttn4Warps; ++x) m = fmaxf(m, parts[x * kRingFloats + kRows * kPitch + row]);
#pragma unroll
    for (int x = 0; x < kAttn4Warps; ++x) {
      const float mw = parts[x * kRingFloats + kRows * kPitch + row];
      const float f = mw == -INFINITY ? 0.f : ex2_approx(mw - m);
      const float lw = parts[x * kRingFloats + kRows * kPitch + kRows + row];
      if (mw != -INFINITY || lw != 0.f) {  // NaN sums are kept
        lsum += f * lw;
        acc = fmaf(f, parts[x * kRingFloats + row * kPitch + ch], acc);
      }
    }
    joined[row * kPitch + ch] = acc;
    if (ch == 0) {
      joined[kRows * kPitch + row] = m;
      joined[kRows * kPitch + kRows + row] = lsum;
    }
  }
  if (p.splits > 1) cluster_sync_all(); else __syncthreads();
  const uint32_t joined_u = smem_u32(joined);
  for (int row = static_cast<int>(split); row < kRows && row0 + row < rows; row += p.splits) {
    const int ch = threadIdx.x;
    float m = -INFINITY, lsum = 0.f, acc = 0.f;
    for (int x = 0; x < p.splits; ++x) m = fmaxf(m, dsmem_ld(joined_u + (kRows * kPitch + row) * 4, x));
    for (int x = 0; x < p.splits; ++x) {
      const float mw = dsmem_ld(joined_u + (kRows * kPitch + row) * 4, x);
      const float lw = dsmem_ld(joined_u + (kRows * kPitch + kRows + row) * 4, x);
      const float f = mw == -INFINITY ? 0.f : ex2_approx(mw - m);
      if (mw != -INFINITY || lw != 0.f) {
        lsum += f * lw;
        acc = fmaf(f, dsmem_ld(joined_u + (row * kPitch + ch) * 4, x), acc);
      }
    }
    const int rr = row0 + row;
    const int tok = rr / p.group;
    const int head = kvh * p.group + rr - tok * p.group;
    const float res = lsum == 0.f ? 0.f : acc / lsum;
    p.out[((q0 + static_cast<int64_t>(tok)) * p.heads_q + head) * 128 + ch] = __float2bfloat16(res);
    if (ch == 0)  // l carries the bias 2^8 of P
      p.lse[head * p.total_q + q0 + tok] =
          lsum == 0.f ? -INFINITY : (m + lg2_approx(lsum) - kAttn4PBias) * 0.69314718055994531f;
  }
  if (p.splits > 1) cluster_sync_all();  // no block leaves while another reads its partial
}

template <int kTiles> constexpr uint32_t attn4_smem_bytes() {
  return kAttn4Warps * kAttn4Ring + (8 * kTiles * 132 + 16 * kTiles) * 4;
}

}  // namespace lpfa
