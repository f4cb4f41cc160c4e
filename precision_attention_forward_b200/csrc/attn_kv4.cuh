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
//
// Range. P is FP16 with the bias 2^10, relative to a reference that trails the maximum by at most 2^4. V's
// scale is an FP16 power of two relative to a unit, one for each of the four channel blocks, which the
// warp takes from its first tile; the window of scales from 2^-15 to 2^0 of the unit becomes 2^-14 to 2^1,
// and the product of both is at most 2^15. A weight keeps its 11 bits down to 2^-24 of the reference, and
// its product down to 2^-25 of the largest that the window allows; below that a product is off by at most
// 2^-35 of the reference times the unit: 2^-20 of the row's largest p 2^e (e: the scale) at worst, since
// the key of the reference has a scale in the window too. With a scale outside the window neither holds: a
// large one that the row does not see or hardly weighs would take the others' bits. From such a tile on,
// the warp joins P and V's scale in FP32 and rounds once, relative to the tile's largest p 2^e in each row
// and channel block (attn4_wide). That costs up to 1.8 times the tame form: 64 ragged sequences of up to
// 8192 keys with scales over 30 binades at random take 118 instead of 69 us. O is FP32 in the block's
// unit, with room for 2^60 above it, where the unit moves, and 2^100 below. S and the softmax statistics
// are FP32.
//
// Split. Each warp of a block walks its own tiles of 32 keys with its own running maximum and accumulators
// (no barrier in the loop); the tiles ahead come by bulk copies into the warp's ring, four for a tile
// within one page, from one lane, and eight, from two, for the halves of a tile of 16-token pages. What
// the lanes of a row or column share, they compute once: lane i turns key i's scale bytes into factors and
// leaves them in shared memory. The blocks of a cluster share the keys of one (sequence, key head, query
// tile) and join their partial results through distributed shared memory: one launch, no workspace, and
// always the same order of sums.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "kv4.cuh"
#include "ptx.cuh"

namespace lpfa {

// Warps of a block: 16 of them on an SM at 128 registers (8 query rows), 8 at twice as many (16 rows).
template <int kTiles> constexpr int attn4_warps() { return kTiles == 1 ? 8 : 4; }
constexpr int kAttn4Keys = 32;                 // keys of a warp's tile
constexpr int kAttn4Stages = 3;                // tiles per warp in shared memory
constexpr int kAttn4StageBytes = kAttn4Keys * (64 + 64 + 4 + 4);  // K, V, their scale words
// A warp's shared memory: the ring, the factors of K (4 floats a key) and of V (4 halves a key), and the
// ring's barriers.
constexpr int kAttn4KFactors = kAttn4Stages * kAttn4StageBytes;
constexpr int kAttn4VFactors = kAttn4KFactors + kAttn4Keys * 16;
constexpr int kAttn4Bars = kAttn4VFactors + kAttn4Keys * 8;
constexpr int kAttn4Ring = kAttn4Bars + 16 * ((kAttn4Stages + 1) / 2);
constexpr int kAttn4MaxSplit = 16;  // blocks of a cluster
constexpr int kAttn4SortRounds = 4;  // rounds of blocks up to which the sequences are put in order
constexpr int kAttn4SortKeys = 1024;  // keys of the longest one from which on they are
constexpr float kAttn4Lag = 4.f;    // binades that the running maximum may be exceeded by
constexpr int kAttn4PBias = 10;     // P is 2^10 e^(s - m), at most 2^14
constexpr int kAttn4VBias = 1;      // V's scale is 2^(1 + byte - unit), at most 2^1
constexpr int kAttn4VRoom = 4;      // the unit is the first tile's largest byte and this much more, for the tiles after it
constexpr int kAttn4VAbove = 60;    // a byte further above the unit moves it

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
  int sorted;  // take the sequences in order of their lengths
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
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zero.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
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

// The units of V's scales in channel blocks 0 and 2 (word 0) or 1 and 3 (word 1) as a packed addend: byte +
// (15 - unit) is a byte's place in the window, 0 to 15.
__device__ __forceinline__ uint32_t v_addend(int unit_lo, int unit_hi) {
  return static_cast<uint32_t>(15 - unit_lo) + (static_cast<uint32_t>(15 - unit_hi) << 16);
}
__device__ __forceinline__ void v_units(uint32_t addend, int& unit_lo, int& unit_hi) {
  const int lo = static_cast<int16_t>(addend & 0xFFFFu);
  unit_lo = 15 - lo;
  unit_hi = 15 - (static_cast<int32_t>(addend - static_cast<uint32_t>(lo)) >> 16);
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

// Physical key of row m (0..7) of an 8-row half of a fragment: 0 5 1 4 2 7 3 6. With it the eight rows
// that a quarter warp reads for K fall into different banks, and V's reads take two passes for four.
__device__ __forceinline__ int attn4_key(int m) { return (m & 1) ? 4 + ((m >> 1) ^ 1) : m >> 1; }
// And back: the row of the fragment that holds key k (0..7).
__device__ __forceinline__ int attn4_row(int k) { return k < 4 ? 2 * k : 2 * ((k - 4) ^ 1) + 1; }

// The softmax and O^T += V^T P^T of a tile where V's scales lie far apart (see the head of the file): with z
// the exponent of P, the weight of a key in a channel block is 2^(z + byte + kAttn4VBias - unit), and goes in
// relative to the tile's largest one in its row. Rare, so short before fast.
template <int kTiles>
__device__ __forceinline__ void attn4_wide(const uint8_t* kt, int lane, const uint32_t (&vadd)[2],
                                           float (&s)[2][kTiles][4], const float (&c2)[kTiles][2],
                                           const float (&off)[kTiles][2], float (&l)[kTiles][2],
                                           float (&o)[kTiles][8][4]) {
  constexpr float kTop = 14.f;  // the largest weight goes in as 2^14
  const uint8_t* vt = kt + 2048;
  const int g = lane >> 2, t = lane & 3;
  int unit[4];
  v_units(vadd[0], unit[0], unit[2]);
  v_units(vadd[1], unit[1], unit[3]);
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[h][n][i] = fmaf(s[h][n][i], c2[n][i & 1], off[n][i & 1]);
        l[n][i & 1] += ex2_approx(s[h][n][i]);
      }
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    float by[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        by[h][e] = static_cast<float>(static_cast<int>(kt[4224 + 4 * (16 * h + 8 * e + attn4_key(g)) + b]) + kAttn4VBias - unit[b]);
    uint32_t pw[2][kTiles][2];
    float back[kTiles][2];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      float low[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float m = fmaxf(fmaxf(s[0][n][i] + by[0][0], s[0][n][2 + i] + by[0][1]),
                        fmaxf(s[1][n][i] + by[1][0], s[1][n][2 + i] + by[1][1]));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
        back[n][i] = ex2_approx(m - kTop);
        low[i] = m == -INFINITY ? 0.f : kTop - m;  // no key of the tile: every weight is 2^-inf
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float a0 = by[h][0], a1 = by[h][1];
        pw[h][n][0] = movmatrix(half2_bits(ex2_approx(s[h][n][0] + (a0 + low[0])), ex2_approx(s[h][n][1] + (a0 + low[1]))));
        pw[h][n][1] = movmatrix(half2_bits(ex2_approx(s[h][n][2] + (a1 + low[0])), ex2_approx(s[h][n][3] + (a1 + low[1]))));
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t a[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // Byte 2 b + j of the eight of a key that this lane's fragment holds: the codes of two channels.
        const uint8_t* ra = vt + (16 * h + t) * 64 + g * 8 + 2 * b + j;
        const uint8_t* rb = vt + (16 * h + 4 + (t ^ 1)) * 64 + g * 8 + 2 * b + j;
        const uint32_t wa = ra[0], wb = rb[0], wc = ra[512], wd = rb[512];
        a[h][0] = cvt_e2m1x2_to_f16x2<0>((wa & 0xFu) | (wb << 4));
        a[h][1] = cvt_e2m1x2_to_f16x2<0>((wa >> 4) | (wb & 0xF0u));
        a[h][2] = cvt_e2m1x2_to_f16x2<0>((wc & 0xFu) | (wd << 4));
        a[h][3] = cvt_e2m1x2_to_f16x2<0>((wc >> 4) | (wd & 0xF0u));
      }
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        float d[4];
        mma_f16_zero(d, a[0][0], a[0][1], a[0][2], a[0][3], pw[0][n][0], pw[0][n][1]);
        mma_f16(d, a[1][0], a[1][1], a[1][2], a[1][3], pw[1][n][0], pw[1][n][1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][2 * b + j][i] = fmaf(d[i], back[n][i & 1], o[n][2 * b + j][i]);
      }
    }
  }
}

// Sequence number `nth` of the lengths in falling order, to a 64th of the longest, and equals by their number; where
// all are short, just number `nth`. Every block works it out for itself, since the lengths are on the device only,
// with work in proportion to their number, about 1 us a block for a few hundred. All threads take part; `mem`
// holds 64 + 2 kWarps words.
template <int kWarps>
__device__ __forceinline__ int attn4_nth_longest(const int32_t* lens, int n, int nth, int32_t* mem) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t *count = mem, *tops = mem + 64, *found = tops + kWarps;
  int top = 1;
  for (int i = threadIdx.x; i < n; i += 32 * kWarps) top = max(top, __ldg(lens + i));
  top = __reduce_max_sync(kAll, top);
  if (lane == 0) tops[warp] = top;
  if (threadIdx.x < 64) count[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = max(top, tops[w]);
  if (top < kAttn4SortKeys) return nth;
  const float scale = 63.5f / static_cast<float>(top);
  auto bucket = [&](int i) { return 63 - static_cast<int>(scale * static_cast<float>(max(0, __ldg(lens + i)))); };
  for (int i = threadIdx.x; i < n; i += 32 * kWarps) atomicAdd(&count[bucket(i)], 1);
  __syncthreads();
  // The bucket that holds number nth, and its number there: lane's two buckets start at number `before`.
  const int c0 = count[2 * lane], c1 = count[2 * lane + 1];
  int before = c0 + c1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(kAll, before, d);
    if (lane >= d) before += up;
  }
  before -= c0 + c1;
  const int owner = 31 - __clz(__ballot_sync(kAll, before <= nth));
  const int second = nth >= before + c0;
  const int mine = __shfl_sync(kAll, 2 * lane + second, owner);
  int left = nth - __shfl_sync(kAll, before + (second ? c0 : 0), owner);
  // Each warp counts the bucket's members in a part of the sequences; then the part that has it is gone through.
  const int part = (n + 32 * kWarps - 1) / (32 * kWarps) * 32;
  int members = 0;
  for (int i = warp * part; i < min(n, (warp + 1) * part); i += 32)
    members += __popc(__ballot_sync(kAll, i + lane < n && bucket(i + lane) == mine));
  if (lane == 0) found[warp] = members;
  __syncthreads();
  int at = 0;
  for (; at < kWarps - 1 && left >= found[at]; ++at) left -= found[at];
  for (int i = at * part;; i += 32) {
    const uint32_t in = __ballot_sync(kAll, i + lane < n && bucket(i + lane) == mine);
    if (left >= __popc(in) && i + 32 < n) {
      left -= __popc(in);
      continue;
    }
    const uint32_t it = __ballot_sync(kAll, ((in >> lane) & 1u) && __popc(in & ((1u << lane) - 1u)) == left);
    return max(0, i + __ffs(it) - 1);
  }
}

// kTiles: tiles of 8 query rows that a block holds (rows = query tokens x query heads of a key head).
template <int kTiles>
__global__ void __launch_bounds__(32 * attn4_warps<kTiles>(), kTiles == 1 ? 16 / attn4_warps<kTiles>() : 2)
attn_kv4_kernel(const __grid_constant__ Attn4Params p) {
  constexpr int kAttn4Warps = attn4_warps<kTiles>();
  constexpr int kAttn4Threads = 32 * kAttn4Warps;
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
  int seq = w / p.c.heads;
  if (p.sorted) {
    // Longest sequences first, so that the last blocks to run are short ones.
    seq = attn4_nth_longest<kAttn4Warps>(p.kv_lens, p.num_seqs, seq, reinterpret_cast<int32_t*>(smem4));
    __syncthreads();  // the rings come next in this memory
  }
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
  // Reference, offset of the exponent (0 while every s is -inf), sum of P.
  float mx[kTiles][2], off[kTiles][2], l[kTiles][2];
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][d][i] = 0.f;
    mx[n][0] = mx[n][1] = -INFINITY;
    off[n][0] = off[n][1] = 0.f;
    l[n][0] = l[n][1] = 0.f;
  }
  constexpr int kNoUnit = -16384;  // the first tile finds every byte far above its unit
  uint32_t vadd[2] = {v_addend(kNoUnit, kNoUnit), v_addend(kNoUnit, kNoUnit)};

  uint8_t* ring = smem4 + warp * kAttn4Ring;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + kAttn4Bars);
  if (lane == 0) {
    for (int i = 0; i < kAttn4Stages; ++i) mbar_init(&bars[i], 1);
    mbar_fence_init();
  }
  __syncwarp();
  // Table entries of the two 16-key halves of a tile; -1 beyond hi.
  const int32_t* table = p.c.table + seq * p.c.table_stride;
  const bool whole = p.c.page_shift >= 5;  // a tile lies within one page
  auto entries = [&](int tile) {
    const int key = tile * kAttn4Keys;
    if (whole) return make_int2(key < hi ? __ldg(table + (key >> p.c.page_shift)) : -1, 0);
    return make_int2(key < hi ? __ldg(table + (key >> p.c.page_shift)) : -1,
                     key + 16 < hi ? __ldg(table + ((key + 16) >> p.c.page_shift)) : -1);
  };
  // Tile `tile`, whose entries are `pg`, into ring stage `st`: whole halves, of pages that are in the pool.
  // Returns the halves (bits 0 and 1) that have keys but no such page: those keys are not seen.
  const uint32_t leader = lane == 0;
  auto load_tile = [&](int tile, int2 pg, int st) {
    uint8_t* dst = ring + st * kAttn4StageBytes;
    const int key0 = tile * kAttn4Keys;
    const bool has0 = static_cast<uint32_t>(pg.x) < static_cast<uint32_t>(p.c.pages);
    const int64_t row0 = ((static_cast<int64_t>(pg.x) * p.c.heads + kvh) << p.c.page_shift) + (key0 & (p.c.page_size - 1));
    fence_proxy_async_smem();  // the lanes' reads of the stage precede its next copies
    if (whole) {
      mbar_arrive_expect_tx(&bars[st], has0 ? kAttn4StageBytes : 0, leader);
      if (has0) {
        bulk_load(dst, p.c.payload[0] + row0 * 64, 2048, &bars[st], leader);
        bulk_load(dst + 2048, p.c.payload[1] + row0 * 64, 2048, &bars[st], leader);
        bulk_load(dst + 4096, p.c.scales[0] + row0 * 4, 128, &bars[st], leader);
        bulk_load(dst + 4224, p.c.scales[1] + row0 * 4, 128, &bars[st], leader);
        return 0u;
      }
      if (lane == 0) kv4_bad_entry(kKv4AttnPageSite);
      return 3u;
    }
    const bool has1 = static_cast<uint32_t>(pg.y) < static_cast<uint32_t>(p.c.pages);
    const int64_t row1 =
        ((static_cast<int64_t>(pg.y) * p.c.heads + kvh) << p.c.page_shift) + ((key0 + 16) & (p.c.page_size - 1));
    mbar_arrive_expect_tx(&bars[st], (kAttn4StageBytes / 2) * (has0 + has1), leader);
    // Lanes 0 and 1 fetch a half each.
    const uint32_t fetch = lane == 0 ? has0 : lane == 1 ? has1 : 0u;
    const int64_t row = lane ? row1 : row0;
    bulk_load(dst + 1024 * lane, p.c.payload[0] + row * 64, 1024, &bars[st], fetch);
    bulk_load(dst + 2048 + 1024 * lane, p.c.payload[1] + row * 64, 1024, &bars[st], fetch);
    bulk_load(dst + 4096 + 64 * lane, p.c.scales[0] + row * 4, 64, &bars[st], fetch);
    bulk_load(dst + 4224 + 64 * lane, p.c.scales[1] + row * 4, 64, &bars[st], fetch);
    const uint32_t missing = (key0 < hi && !has0 ? 1u : 0u) | (key0 + 16 < hi && !has1 ? 2u : 0u);
    if (missing && lane == 0) kv4_bad_entry(kKv4AttnPageSite);
    return missing;
  };

  const int mine = tile0 + warp;  // this warp's tiles: mine, mine + kAttn4Warps, ...
  uint32_t bad = 0;  // two bits per stage: halves whose page is missing
#pragma unroll
  for (int st = 0; st < kAttn4Stages - 1; ++st) {
    const int tile = mine + st * kAttn4Warps;
    if (tile < tile1) bad |= load_tile(tile, entries(tile), st) << (2 * st);
  }
  // Where lane i leaves key i's factors, and where a lane finds those of its fragment's keys.
  float4* kfac = reinterpret_cast<float4*>(ring + kAttn4KFactors);
  uint8_t* vfac = ring + kAttn4VFactors;  // [tile of 16][pair t][half of 8][block] half2 (keys 2t, 2t + 1)
  uint16_t* vfac_mine;
  {
    const int m = attn4_row(lane & 7);
    vfac_mine = reinterpret_cast<uint16_t*>(vfac + (((lane >> 4) * 4 + (m >> 1)) * 2 + ((lane >> 3) & 1)) * 16) + (m & 1);
  }
  int st = 0;
  uint32_t phase = 0;
  int2 ahead = entries(mine + (kAttn4Stages - 1) * kAttn4Warps);  // loaded a tile before they are needed
  // The steps of a tile. Refill of the stage before it, and the wait for its own; false: the wait ran out.
  auto fetch = [&](int tile) {
    __syncwarp();  // the stage to refill, and the factors, have been read
    const int next = tile + (kAttn4Stages - 1) * kAttn4Warps;
    const int nst = st == 0 ? kAttn4Stages - 1 : st - 1;
    bad &= ~(3u << (2 * nst));
    if (next < tile1) bad |= load_tile(next, ahead, nst) << (2 * nst);
    ahead = entries(next + kAttn4Warps);
    if (mbar_wait(&bars[st], phase, nullptr)) return true;
    if (atomicCAS(&g_lpfa_status[0], 0, 4 /* LPFA_ERR_TIMEOUT */) == 0) atomicExch(&g_lpfa_status[1], kKv4AttnWaitSite);
    // Every copy under way has to land before this memory is used again or the block ends (bounded too).
    for (int k = 0; k < kAttn4Stages && tile + k * kAttn4Warps < tile1; ++k)
      mbar_wait(&bars[(st + k) % kAttn4Stages], phase ^ (st + k >= kAttn4Stages ? 1u : 0u), nullptr);
    return false;
  };
  // Scale words of key `lane`, K's as factors into shared memory (2^e as floats; byte 0, 2^-127, counts as 0). Those of
  // a key beyond hi or without a page may be anything: its scores are masked.
  auto scale_words = [&]() {
    const uint8_t* kt = ring + st * kAttn4StageBytes;
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(kt + 4096 + 4 * lane);
    kfac[lane] = make_float4(__uint_as_float((kw << 23) & 0x7F800000u), __uint_as_float((kw << 15) & 0x7F800000u),
                             __uint_as_float((kw << 7) & 0x7F800000u), __uint_as_float((kw >> 1) & 0x7F800000u));
    return *reinterpret_cast<const uint32_t*>(kt + 4224 + 4 * lane);
  };
  auto is_there = [&](int tile) { return tile * kAttn4Keys + lane < hi && !((bad >> (2 * st + (lane >> 4))) & 1u); };
  // The first tile sets V's units; later a byte far above them moves them, and O with them.
  auto move_units = [&](uint32_t vw) {
    int unit[4];
    v_units(vadd[0], unit[0], unit[2]);
    v_units(vadd[1], unit[1], unit[3]);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int high = static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, (vw >> (8 * b)) & 0xFFu));
      if (high <= unit[b] + kAttn4VAbove) continue;
      const int down = unit[b] - high - kAttn4VRoom;
      const float fv = down < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + down) << 23);
      unit[b] -= down;
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int d = 2 * b; d < 2 * b + 2; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][d][i] *= fv;
    }
    vadd[0] = v_addend(unit[0], unit[2]);
    vadd[1] = v_addend(unit[1], unit[3]);
  };
  // S^T (two tiles of 16 keys): c0, c1: key attn4_key(g), c2, c3: 8 more; columns 2t, 2t + 1.
  auto scores = [&](float (&s)[2][kTiles][4]) {
    const uint8_t* kt = ring + st * kAttn4StageBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r0 = 16 * h + attn4_key(g);
      const uint4 k0 = *reinterpret_cast<const uint4*>(kt + r0 * 64 + t * 16);
      const uint4 k1 = *reinterpret_cast<const uint4*>(kt + (r0 + 8) * 64 + t * 16);
      const float4 f0 = kfac[r0], f1 = kfac[r0 + 8];
      const float x0[4] = {f0.x, f0.y, f0.z, f0.w}, x1[4] = {f1.x, f1.y, f1.z, f1.w};
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
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          float d[4];
          mma_f16_zero(d, a[0][0], a[0][1], a[0][2], a[0][3], qf[n][b][0], qf[n][b][1]);
          mma_f16(d, a[1][0], a[1][1], a[1][2], a[1][3], qf[n][b][2], qf[n][b][3]);
          if (b == 0) {
            s[h][n][0] = d[0] * x0[0];
            s[h][n][1] = d[1] * x0[0];
            s[h][n][2] = d[2] * x1[0];
            s[h][n][3] = d[3] * x1[0];
          } else {
            s[h][n][0] = fmaf(d[0], x0[b], s[h][n][0]);
            s[h][n][1] = fmaf(d[1], x0[b], s[h][n][1]);
            s[h][n][2] = fmaf(d[2], x1[b], s[h][n][2]);
            s[h][n][3] = fmaf(d[3], x1[b], s[h][n][3]);
          }
        }
      }
    }
  };
  // Masks, running maximum (in log2 units: the factor is positive, so it can follow the maximum).
  auto settle = [&](int tile, uint32_t gone, float (&s)[2][kTiles][4]) {
    if (gone != 0 || (tile + 1) * kAttn4Keys > lim_min) {
      const int key0 = tile * kAttn4Keys + attn4_key(g);
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key0 + 16 * h + 8 * (i >> 1) >= lim[n][i & 1] || ((gone >> h) & 1u)) s[h][n][i] = -INFINITY;
    }
    // The reference m follows the maximum only when a key is more than 2^kAttn4Lag above it: until then a
    // lane needs to know its own keys' maximum alone, and no shuffles.
    bool moved = false;
    float top[kTiles][2];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[n][i] = c2[n][i] * fmaxf(fmaxf(s[0][n][i], s[0][n][2 + i]), fmaxf(s[1][n][i], s[1][n][2 + i]));
        moved |= top[n][i] > mx[n][i] + kAttn4Lag;
      }
    }
    if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float m = fmaxf(mx[n][i], top[n][i]);
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
          const float f = mx[n][i] == -INFINITY ? 0.f : ex2_approx(mx[n][i] - m);  // no key yet: o and l are 0
          mx[n][i] = m;
          off[n][i] = m == -INFINITY ? 0.f : static_cast<float>(kAttn4PBias) - m;
          l[n][i] *= f;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            o[n][d][i] *= f;
            o[n][d][2 + i] *= f;
          }
        }
      }
    }
  };
  auto advance = [&]() {
    if (++st == kAttn4Stages) {
      st = 0;
      phase ^= 1u;
    }
  };

  int tile = mine;
#pragma unroll 1
  for (; tile < tile1; tile += kAttn4Warps) {
    if (!fetch(tile)) {
      tile = tile1;
      break;
    }
    const uint8_t* vt = ring + st * kAttn4StageBytes + 2048;
    const uint32_t gone = (bad >> (2 * st)) & 3u;
    {
      const uint32_t vw = scale_words();
      // V: the place in the window of its scales, plus one, is the exponent field of an f16 factor. (A key that
      // is not there has P = 0, and any factor that is finite.)
      const uint32_t v02 = vw & 0x00FF00FFu, v13 = (vw >> 8) & 0x00FF00FFu;
      uint32_t f02 = v02 + vadd[0], f13 = v13 + vadd[1];
      const auto outside = [&]() { return __any_sync(0xFFFFFFFFu, ((f02 | f13) & 0xFFF0FFF0u) != 0u); };
      if (outside()) {
        const bool there = is_there(tile);
        move_units(there ? vw : 0u);
        f02 = there ? v02 + vadd[0] : 0u;
        f13 = there ? v13 + vadd[1] : 0u;
        if (outside()) break;
      }
      f02 = f02 * 1024u + 0x04000400u;
      f13 = f13 * 1024u + 0x04000400u;
      vfac_mine[0] = static_cast<uint16_t>(f02);
      vfac_mine[2] = static_cast<uint16_t>(f13);
      vfac_mine[4] = static_cast<uint16_t>(f02 >> 16);
      vfac_mine[6] = static_cast<uint16_t>(f13 >> 16);
      __syncwarp();
    }
    float s[2][kTiles][4];
    scores(s);
    settle(tile, gone, s);
    // ---- P^T as the B operand: 2^10 e^(s - m), keys 2t, 2t + 1 (and 8 more) of column g
    uint32_t pb[2][kTiles][2];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const float r0 = off[n][0], r1 = off[n][1];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float e0 = ex2_approx(fmaf(s[h][n][0], c2[n][0], r0)), e1 = ex2_approx(fmaf(s[h][n][1], c2[n][1], r1));
        const float e2 = ex2_approx(fmaf(s[h][n][2], c2[n][0], r0)), e3 = ex2_approx(fmaf(s[h][n][3], c2[n][1], r1));
        l[n][0] += e0 + e2;
        l[n][1] += e1 + e3;
        pb[h][n][0] = movmatrix(half2_bits(e0, e1));
        pb[h][n][1] = movmatrix(half2_bits(e2, e3));
      }
    }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // Physical keys of fragment keys 2t, 2t + 1 (and 2t + 8, 2t + 9: 8 more).
      const uint8_t* ra = vt + (16 * h + t) * 64 + g * 8;
      const uint8_t* rb = vt + (16 * h + 4 + (t ^ 1)) * 64 + g * 8;
      const uint2 va = *reinterpret_cast<const uint2*>(ra), vb = *reinterpret_cast<const uint2*>(rb);
      const uint2 vc = *reinterpret_cast<const uint2*>(ra + 512), vd = *reinterpret_cast<const uint2*>(rb + 512);
      const uint4 fab = *reinterpret_cast<const uint4*>(vfac + ((h * 4 + t) * 2) * 16);
      const uint4 fcd = *reinterpret_cast<const uint4*>(vfac + ((h * 4 + t) * 2 + 1) * 16);
      const uint32_t sab[4] = {fab.x, fab.y, fab.z, fab.w}, scd[4] = {fcd.x, fcd.y, fcd.z, fcd.w};
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // blocks 2 half, 2 half + 1
        const uint32_t wa = half ? va.y : va.x, wb = half ? vb.y : vb.x;
        const uint32_t wc = half ? vc.y : vc.x, wd = half ? vd.y : vd.x;
        // Bytes of (first key's, second key's) codes: of the even elements, of the odd ones.
        const uint32_t e0 = (wa & 0x0F0F0F0Fu) | ((wb << 4) & 0xF0F0F0F0u);
        const uint32_t o0 = ((wa >> 4) & 0x0F0F0F0Fu) | (wb & 0xF0F0F0F0u);
        const uint32_t e1 = (wc & 0x0F0F0F0Fu) | ((wd << 4) & 0xF0F0F0F0u);
        const uint32_t o1 = ((wc >> 4) & 0x0F0F0F0Fu) | (wd & 0xF0F0F0F0u);
        uint32_t a[4][4];  // [byte][fragment register]
        a[0][0] = cvt_e2m1x2_to_f16x2<0>(e0); a[0][1] = cvt_e2m1x2_to_f16x2<0>(o0);
        a[0][2] = cvt_e2m1x2_to_f16x2<0>(e1); a[0][3] = cvt_e2m1x2_to_f16x2<0>(o1);
        a[1][0] = cvt_e2m1x2_to_f16x2<1>(e0); a[1][1] = cvt_e2m1x2_to_f16x2<1>(o0);
        a[1][2] = cvt_e2m1x2_to_f16x2<1>(e1); a[1][3] = cvt_e2m1x2_to_f16x2<1>(o1);
        a[2][0] = cvt_e2m1x2_to_f16x2<2>(e0); a[2][1] = cvt_e2m1x2_to_f16x2<2>(o0);
        a[2][2] = cvt_e2m1x2_to_f16x2<2>(e1); a[2][3] = cvt_e2m1x2_to_f16x2<2>(o1);
        a[3][0] = cvt_e2m1x2_to_f16x2<3>(e0); a[3][1] = cvt_e2m1x2_to_f16x2<3>(o0);
        a[3][2] = cvt_e2m1x2_to_f16x2<3>(e1); a[3][3] = cvt_e2m1x2_to_f16x2<3>(o1);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int b = 2 * half + k;
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            const uint32_t p0 = half2_mul(pb[h][n][0], sab[b]), p1 = half2_mul(pb[h][n][1], scd[b]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              mma_f16(o[n][2 * b + j], a[2 * k + j][0], a[2 * k + j][1], a[2 * k + j][2], a[2 * k + j][3], p0, p1);
          }
        }
      }
    }
    advance();
  }
  // From a tile with a scale outside the window on (its keys' scale words are in place).
  if (tile < tile1) {
#pragma unroll 1
    for (;;) {
      __syncwarp();
      float s[2][kTiles][4];
      scores(s);
      settle(tile, (bad >> (2 * st)) & 3u, s);
      attn4_wide<kTiles>(ring + st * kAttn4StageBytes, lane, vadd, s, c2, off, l, o);
      advance();
      tile += kAttn4Warps;
      if (tile >= tile1 || !fetch(tile)) break;
      const uint32_t vw = scale_words();
      move_units(is_there(tile) ? vw : 0u);
    }
  }
  __syncwarp();

  // ---- join: the warp's partial (O without its bias, m, l) over its own ring, then the block's, then
  // the cluster's. Rows that do not exist are left out.
  const int real = min(kRows, rows - row0);
  float* part = reinterpret_cast<float*>(ring);  // [kRows][kPitch], then m[kRows], l[kRows]
  // O is still in V's units and with both biases, l with P's: factors 2^(unit - 127 - biases) in two halves, each a
  // normal number (without a tile there is no unit, and O is 0).
  float undo[4][2];
  {
    int unit[4];
    v_units(vadd[0], unit[0], unit[2]);
    v_units(vadd[1], unit[1], unit[3]);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int e = max(-250, unit[b] - 127 - kAttn4VBias - kAttn4PBias);
      undo[b][0] = __uint_as_float(static_cast<uint32_t>(127 + e / 2) << 23);
      undo[b][1] = __uint_as_float(static_cast<uint32_t>(127 + e - e / 2) << 23);
    }
  }
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 4);
      l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 8);
      l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 16);
      const int row = 8 * n + 2 * t + i;
      if (row >= real) continue;
      if (g == 0) {
        part[kRows * kPitch + row] = mx[n][i];
        part[kRows * kPitch + kRows + row] = l[n][i] * (1.f / (1 << kAttn4PBias));
      }
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        float* to = part + row * kPitch + 32 * (d >> 1) + 4 * g + 2 * (d & 1);
        to[0] = o[n][d][i] * undo[d >> 1][0] * undo[d >> 1][1];
        to[1] = o[n][d][2 + i] * undo[d >> 1][0] * undo[d >> 1][1];
      }
    }
  }
  __syncthreads();
  constexpr int kRingFloats = kAttn4Ring / 4;
  const float* parts = reinterpret_cast<const float*>(smem4);
  // Like a warp's partial; behind the first warp's in its ring, or (16 rows) behind all rings.
  float* joined = reinterpret_cast<float*>(smem4) +
                  (kTiles == 1 ? kRows * (kPitch + 2) : kAttn4Warps * kRingFloats);
  static_assert(kAttn4Warps <= kAttn4MaxSplit && 2 * 8 * (kPitch + 2) * 4 <= kAttn4Ring, "partials fit");
  const int ch = threadIdx.x & 127;
  constexpr int kJoiners = kAttn4Threads / 128;  // threads that join the rows of a channel
  // Sums of the partials x < n of a row, weighted to their largest m. A partial without keys (m = -inf)
  // has l = 0 and counts for nothing, unless its l is NaN.
  auto join = [&](const auto& ms, const auto& ls, const auto& os, int n, float& m, float& lsum, float& acc) {
    constexpr int kMost = sizeof(ms) / sizeof(float);
    m = -INFINITY;
#pragma unroll
    for (int x = 0; x < kMost; ++x)
      if (x < n) m = fmaxf(m, ms[x]);
    lsum = 0.f;
    acc = 0.f;
#pragma unroll
    for (int x = 0; x < kMost; ++x) {
      if (x >= n || (ms[x] == -INFINITY && ls[x] == 0.f)) continue;
      const float f = ms[x] == -INFINITY ? 0.f : ex2_approx(ms[x] - m);
      lsum = fmaf(f, ls[x], lsum);
      acc = fmaf(f, os[x], acc);
    }
  };
  auto finish = [&](int row, float m, float lsum, float acc) {
    const int rr = row0 + row;
    const int tok = rr / p.group;
    const int head = kvh * p.group + rr - tok * p.group;
    const float res = lsum == 0.f ? 0.f : acc / lsum;
    p.out[((q0 + static_cast<int64_t>(tok)) * p.heads_q + head) * 128 + ch] = __float2bfloat16(res);
    if (ch == 0)
      p.lse[head * p.total_q + q0 + tok] =
          lsum == 0.f ? -INFINITY : (m + lg2_approx(lsum)) * 0.69314718055994531f;
  };
  for (int row = threadIdx.x >> 7; row < real; row += kJoiners) {
    float ms[kAttn4Warps], ls[kAttn4Warps], os[kAttn4Warps], m, lsum, acc;
#pragma unroll
    for (int x = 0; x < kAttn4Warps; ++x) {
      ms[x] = parts[x * kRingFloats + kRows * kPitch + row];
      ls[x] = parts[x * kRingFloats + kRows * kPitch + kRows + row];
      os[x] = parts[x * kRingFloats + row * kPitch + ch];
    }
    join(ms, ls, os, kAttn4Warps, m, lsum, acc);
    if (p.splits == 1) {
      finish(row, m, lsum, acc);
    } else {
      joined[row * kPitch + ch] = acc;
      if (ch == 0) {
        joined[kRows * kPitch + row] = m;
        joined[kRows * kPitch + kRows + row] = lsum;
      }
    }
  }
  if (p.splits == 1) return;
  cluster_sync_all();
  const uint32_t joined_u = smem_u32(joined);
  // All of a row's remote reads on the way at once.
  auto join_blocks = [&](auto most) {
    constexpr int kMost = decltype(most)::value;
    for (int row = static_cast<int>(split) + p.splits * (threadIdx.x >> 7); row < real; row += p.splits * kJoiners) {
      float ms[kMost], ls[kMost], os[kMost], m, lsum, acc;
#pragma unroll
      for (int x = 0; x < kMost; ++x) {
        const int from = min(x, p.splits - 1);
        ms[x] = dsmem_ld(joined_u + (kRows * kPitch + row) * 4, from);
        ls[x] = dsmem_ld(joined_u + (kRows * kPitch + kRows + row) * 4, from);
        os[x] = dsmem_ld(joined_u + (row * kPitch + ch) * 4, from);
      }
      join(ms, ls, os, p.splits, m, lsum, acc);
      finish(row, m, lsum, acc);
    }
  };
  if (p.splits <= 4) {
    join_blocks(std::integral_constant<int, 4>{});
  } else if (p.splits <= 8) {
    join_blocks(std::integral_constant<int, 8>{});
  } else {
    join_blocks(std::integral_constant<int, kAttn4MaxSplit>{});
  }
  cluster_sync_all();  // no block leaves while another reads its partial
}

template <int kTiles> constexpr uint32_t attn4_smem_bytes() {
  return attn4_warps<kTiles>() * kAttn4Ring + (kTiles == 1 ? 0 : 16 * 134 * 4);
}

}  // namespace lpfa
