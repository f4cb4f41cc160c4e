// lpfa.cu -- host side of the C ABI declared in include/lpfa.h: argument validation,
// packed varlen metadata, TMA tensor maps and kernel launches. All kernels live in the
// headers included below; this is the library's single translation unit.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <vector>

#include "lpfa.h"
#include "attn_fwd.cuh"
#include "attn_fwd_pp.cuh"
#include "attn_bwd.cuh"
#include "quantize.cuh"
#include "dequantize.cuh"
#include "qk_norm_rope.cuh"
#include "kv4.cuh"
#include "attn_kv4.cuh"

namespace {

thread_local char g_msg[512] = "";

lpfa_status fail(lpfa_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return st;
}

lpfa_status cuda_fail(cudaError_t e, const char* what) {
  return fail(LPFA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  bool init = false;
  bool sm100 = false;
  int sms = 0;
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

// Returns LPFA_OK and fills *info for the current device, or an error status.
lpfa_status current_device(DeviceInfo* info, int* dev_out = nullptr) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(LPFA_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.init) {
    int major = 0, minor = 0, sms = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess)
      return cuda_fail(e, "cudaDeviceGetAttribute");
    if ((e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess)
      return cuda_fail(e, "cudaDeviceGetAttribute");
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return cuda_fail(e, "cudaDeviceGetAttribute");
    d.sm100 = (major == 10 && minor == 0);
    d.sms = sms;
    d.init = true;
  }
  *info = d;
  if (dev_out) *dev_out = dev;
  return LPFA_OK;
}

lpfa_status require_sm100(DeviceInfo* info, int* dev = nullptr) {
  lpfa_status st = current_device(info, dev);
  if (st != LPFA_OK) return st;
  if (!info->sm100) return fail(LPFA_ERR_UNSUPPORTED, "the current device is not sm_100 (B200)");
  return LPFA_OK;
}

// Raises a kernel's dynamic shared memory limit (and allows clusters beyond the portable size) once per
// device: the attributes stay, and setting them costs as much as a tenth of a small call.
struct KernelLimits {
  std::atomic<bool> set[kMaxDevices] = {};
};
lpfa_status set_limits(KernelLimits& k, const void* fn, int dev, int smem, bool clusters) {
  if (k.set[dev].load(std::memory_order_acquire)) return LPFA_OK;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && clusters) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  k.set[dev].store(true, std::memory_order_release);
  return LPFA_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Tensor map over a packed (tokens, heads, 128) uint8 payload; box = box_rows tokens of one
// head, 128-byte rows with the 128-byte swizzle the UMMA descriptors expect.
lpfa_status payload_tmap(CUtensorMap* map, const void* base, int64_t tokens, int heads, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return fail(LPFA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {128, static_cast<cuuint64_t>(heads) * 128};
  cuuint32_t box[3] = {128, 1, box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(LPFA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return LPFA_OK;
}

// Tensor map over a strided (tokens, heads, 128) input of bf16 or fp32 elements; box = 128
// tokens of one head, no swizzle. A dimension of extent 1 gets a dummy stride (it is never
// stepped over).
lpfa_status input_tmap(CUtensorMap* map, const void* base, bool fp32, int64_t tokens, int heads, int64_t tok_stride,
                       int64_t head_stride) {
  auto fn = encode_fn();
  if (!fn) return fail(LPFA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const int64_t es = fp32 ? 4 : 2;
  const int64_t hs = heads > 1 ? head_stride * es : 128 * es;
  const int64_t ts = tokens > 1 ? tok_stride * es : 128 * es * heads;
  if (hs <= 0 || ts <= 0) return fail(LPFA_ERR_INVALID_ARG, "strides must be positive");
  cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(hs), static_cast<cuuint64_t>(ts)};
  cuuint32_t box[3] = {128, 1, 128};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(LPFA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return LPFA_OK;
}

// Tensor map over a contiguous (tokens, heads, 128) BF16 V; box = 64 elements (128 bytes) of
// one head x 128 tokens with the 128-byte swizzle: the two boxes of a 128-key tile are the two
// MN-major swizzle atoms of the BF16 PV operand.
lpfa_status bf16_v_tmap(CUtensorMap* map, const void* base, int64_t tokens, int heads) {
  auto fn = encode_fn();
  if (!fn) return fail(LPFA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {256, static_cast<cuuint64_t>(heads) * 256};
  cuuint32_t box[3] = {64, 1, 128};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(LPFA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return LPFA_OK;
}

lpfa_status check_meta(const lpfa_varlen_meta* m, const char* name) {
  if (!m) return fail(LPFA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!m->dev) return fail(LPFA_ERR_INVALID_ARG, "%s has no device buffer", name);
  if (m->num_seqs < 1 || m->total_tokens < 1 || m->total_scale_blocks < 1)
    return fail(LPFA_ERR_INVALID_ARG, "%s is empty or was not filled", name);
  return LPFA_OK;
}

}  // namespace

extern "C" {

const char* lpfa_last_error_message(void) { return g_msg; }

const char* lpfa_version(void) { return "lpfa 0.1.0 (sm_100a)"; }

size_t lpfa_meta_dev_ints(int32_t num_seqs) {
  return num_seqs < 1 ? 0 : 2 * (static_cast<size_t>(num_seqs) + 1);
}

size_t lpfa_scale_bytes(const lpfa_varlen_meta* meta, int32_t heads) {
  if (!meta || heads < 1 || meta->total_scale_blocks < 0) return 0;
  return static_cast<size_t>(meta->total_scale_blocks) * static_cast<size_t>(heads) * 512u;
}

lpfa_status lpfa_varlen_meta_fill_host(const int32_t* lengths_host, int32_t num_seqs, int32_t* host_ints,
                                       lpfa_varlen_meta* meta) {
  if (!lengths_host || !host_ints || !meta) return fail(LPFA_ERR_INVALID_ARG, "NULL argument");
  if (num_seqs < 1) return fail(LPFA_ERR_INVALID_ARG, "num_seqs must be >= 1 (got %d)", num_seqs);
  int64_t cu = 0, so = 0;
  int32_t mx = 0;
  int32_t* cu_arr = host_ints;
  int32_t* so_arr = host_ints + num_seqs + 1;
  cu_arr[0] = 0;
  so_arr[0] = 0;
  for (int32_t i = 0; i < num_seqs; ++i) {
    const int32_t len = lengths_host[i];
    if (len < 1) return fail(LPFA_ERR_INVALID_ARG, "sequence %d has length %d; lengths must be >= 1", i, len);
    cu += len;
    so += (len + 127) / 128;
    if (cu > INT32_MAX) return fail(LPFA_ERR_INVALID_ARG, "total token count overflows int32");
    cu_arr[i + 1] = static_cast<int32_t>(cu);
    so_arr[i + 1] = static_cast<int32_t>(so);
    if (len > mx) mx = len;
  }
  meta->num_seqs = num_seqs;
  meta->total_tokens = static_cast<int32_t>(cu);
  meta->total_scale_blocks = static_cast<int32_t>(so);
  meta->max_seqlen = mx;
  return LPFA_OK;
}

lpfa_status lpfa_varlen_meta_from_lengths(const int32_t* lengths_host, int32_t num_seqs, lpfa_varlen_meta* meta,
                                          void* stream) {
  if (!meta) return fail(LPFA_ERR_INVALID_ARG, "meta is NULL");
  if (!meta->dev) return fail(LPFA_ERR_INVALID_ARG, "meta->dev must point to a device buffer");
  if (num_seqs < 1) return fail(LPFA_ERR_INVALID_ARG, "num_seqs must be >= 1 (got %d)", num_seqs);
  std::vector<int32_t> host(lpfa_meta_dev_ints(num_seqs));
  lpfa_varlen_meta tmp = *meta;
  lpfa_status st = lpfa_varlen_meta_fill_host(lengths_host, num_seqs, host.data(), &tmp);
  if (st != LPFA_OK) return st;
  // Pageable source: the runtime stages the bytes before returning, so `host` may go away.
  cudaError_t e = cudaMemcpyAsync(meta->dev, host.data(), host.size() * sizeof(int32_t), cudaMemcpyHostToDevice,
                                  static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyAsync(meta)");
  *meta = tmp;
  return LPFA_OK;
}

// Persistent launch of the streaming quantize/cast kernel: as many CTAs as fit on the SMs
// (shared-memory bound), each walking tiles with the grid stride.
static lpfa_status launch_quant(void (*kernel)(const CUtensorMap, lpfa::QuantParams), uint32_t smem, int threads,
                                const CUtensorMap& tmap, const lpfa::QuantParams& p, int sms, cudaStream_t s,
                                const char* what) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  int per_sm = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor");
  if (per_sm < 1) return fail(LPFA_ERR_UNSUPPORTED, "%s: kernel does not fit on an SM", what);
  const int64_t tiles = static_cast<int64_t>(p.num_blocks) * p.heads;
  const int64_t grid = tiles < static_cast<int64_t>(per_sm) * sms ? tiles : static_cast<int64_t>(per_sm) * sms;
  kernel<<<static_cast<unsigned>(grid), threads, smem, s>>>(tmap, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, what);
  return LPFA_OK;
}

// Both orientations of the varlen quantizer: scales along head_dim or along the tokens.
static lpfa_status quantize_impl(const void* x, lpfa_in_dtype dt, int64_t tok_stride, int64_t head_stride,
                                 int32_t heads, int32_t head_dim, const lpfa_varlen_meta* meta,
                                 lpfa_scaling_mode mode, uint8_t* payload, uint8_t* scales, void* stream,
                                 bool tokens) {
  if (!x || !payload || !scales) return fail(LPFA_ERR_INVALID_ARG, "NULL tensor pointer");
  if (dt != LPFA_IN_BF16 && dt != LPFA_IN_FP32) return fail(LPFA_ERR_INVALID_ARG, "invalid input dtype %d", dt);
  if (mode != LPFA_SCALE_RCEIL && mode != LPFA_SCALE_FLOOR) return fail(LPFA_ERR_INVALID_ARG, "invalid scaling mode %d", mode);
  if (head_dim != 128) return fail(LPFA_ERR_INVALID_ARG, "head_dim must be 128 (got %d)", head_dim);
  if (heads < 1) return fail(LPFA_ERR_INVALID_ARG, "heads must be >= 1");
  lpfa_status st = check_meta(meta, "meta");
  if (st != LPFA_OK) return st;
  const int vec = dt == LPFA_IN_BF16 ? 8 : 4;
  if (!aligned16(x) || !aligned16(payload) || (tok_stride % vec) || (head_stride % vec))
    return fail(LPFA_ERR_INVALID_ARG, "x/payload must be 16-byte aligned with strides multiple of %d elements", vec);
  if (!aligned16(scales)) return fail(LPFA_ERR_INVALID_ARG, "scales must be 16-byte aligned");
  DeviceInfo info;
  if ((st = require_sm100(&info)) != LPFA_OK) return st;
  lpfa::QuantParams p = {};
  p.x = x;
  p.tok_stride = tok_stride;
  p.head_stride = head_stride;
  p.heads = heads;
  p.num_seqs = meta->num_seqs;
  p.cu_seqlens = meta->dev;
  p.scale_off = meta->dev + meta->num_seqs + 1;
  p.num_blocks = meta->total_scale_blocks;
  p.payload = payload;
  p.scales = scales;
  p.floor_mode = mode == LPFA_SCALE_FLOOR ? 1 : 0;
  if (static_cast<int64_t>(p.num_blocks) * heads > INT32_MAX) return fail(LPFA_ERR_INVALID_ARG, "too many tiles");
  CUtensorMap tm;
  if ((st = input_tmap(&tm, x, dt == LPFA_IN_FP32, meta->total_tokens, heads, tok_stride, head_stride)) != LPFA_OK)
    return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dt == LPFA_IN_BF16) {
    auto kernel = tokens ? lpfa::quantize_mxfp8_kernel<__nv_bfloat16, lpfa::kQuantTokens>
                         : lpfa::quantize_mxfp8_kernel<__nv_bfloat16, lpfa::kQuantHeadDim>;
    return launch_quant(kernel, lpfa::quant_smem_bytes<__nv_bfloat16>(), lpfa::quant_threads<__nv_bfloat16>(), tm,
                        p, info.sms, s, "quantize launch");
  }
  auto kernel = tokens ? lpfa::quantize_mxfp8_kernel<float, lpfa::kQuantTokens>
                       : lpfa::quantize_mxfp8_kernel<float, lpfa::kQuantHeadDim>;
  return launch_quant(kernel, lpfa::quant_smem_bytes<float>(), lpfa::quant_threads<float>(), tm, p, info.sms, s,
                      "quantize launch");
}

lpfa_status lpfa_quantize_mxfp8_varlen(const void* x, lpfa_in_dtype dt, int64_t tok_stride, int64_t head_stride,
                                       int32_t heads, int32_t head_dim, const lpfa_varlen_meta* meta,
                                       lpfa_scaling_mode mode, uint8_t* payload, uint8_t* scales, void* stream) {
  return quantize_impl(x, dt, tok_stride, head_stride, heads, head_dim, meta, mode, payload, scales, stream, false);
}

lpfa_status lpfa_quantize_mxfp8_varlen_tokens(const void* x, lpfa_in_dtype dt, int64_t tok_stride,
                                              int64_t head_stride, int32_t heads, int32_t head_dim,
                                              const lpfa_varlen_meta* meta, lpfa_scaling_mode mode,
                                              uint8_t* payload, uint8_t* scales, void* stream) {
  return quantize_impl(x, dt, tok_stride, head_stride, heads, head_dim, meta, mode, payload, scales, stream, true);
}

lpfa_status lpfa_cast_e4m3(const void* v_bf16, int64_t tok_stride, int64_t head_stride, int64_t tokens,
                           int32_t heads, int32_t head_dim, uint8_t* out, void* stream) {
  if (!v_bf16 || !out) return fail(LPFA_ERR_INVALID_ARG, "NULL tensor pointer");
  if (head_dim != 128) return fail(LPFA_ERR_INVALID_ARG, "head_dim must be 128 (got %d)", head_dim);
  if (tokens < 1 || heads < 1) return fail(LPFA_ERR_INVALID_ARG, "tokens and heads must be >= 1");
  if (!aligned16(v_bf16) || !aligned16(out) || (tok_stride % 8) || (head_stride % 8))
    return fail(LPFA_ERR_INVALID_ARG, "v/out must be 16-byte aligned with strides multiple of 8 elements");
  DeviceInfo info;
  lpfa_status st = require_sm100(&info);
  if (st != LPFA_OK) return st;
  lpfa::QuantParams p = {};
  p.x = v_bf16;
  p.tok_stride = tok_stride;
  p.head_stride = head_stride;
  p.heads = heads;
  p.tokens = tokens;
  const int64_t blocks = (tokens + 127) / 128;
  if (blocks * heads > INT32_MAX) return fail(LPFA_ERR_INVALID_ARG, "too many tiles");
  p.num_blocks = static_cast<int>(blocks);
  p.payload = out;
  CUtensorMap tm;
  if ((st = input_tmap(&tm, v_bf16, false, tokens, heads, tok_stride, head_stride)) != LPFA_OK) return st;
  return launch_quant(lpfa::quantize_mxfp8_kernel<__nv_bfloat16, lpfa::kQuantCast>, lpfa::quant_smem_bytes<__nv_bfloat16>(),
                        lpfa::quant_threads<__nv_bfloat16>(), tm, p,
                      info.sms, static_cast<cudaStream_t>(stream), "cast launch");
}

// The attention kernel moves registers between its warpgroups with setmaxnreg; the split
// adds up to exactly the launch allocation of kLaunchRegs per thread, so a build whose
// register count differs is refused here instead of launched (a larger split than the
// allocation would never be granted). Also raises the dynamic shared memory limit.
static lpfa_status check_attn_kernel(const void* fn, uint32_t smem_bytes) {
  cudaFuncAttributes attr;
  cudaError_t e = cudaFuncGetAttributes(&attr, fn);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes");
  if (attr.numRegs != lpfa::kLaunchRegs)
    return fail(LPFA_ERR_UNSUPPORTED, "attention kernel built with %d registers per thread; its warpgroup register "
                "split needs exactly %d", attr.numRegs, lpfa::kLaunchRegs);
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem_bytes));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  return LPFA_OK;
}

// MXFP8 (head_dim orientation) -> BF16 over every token of meta: one CTA per (block, head) tile.
static lpfa_status launch_dequant(const uint8_t* payload, const uint8_t* scales, const lpfa_varlen_meta* meta,
                                  int32_t heads, __nv_bfloat16* out, cudaStream_t s) {
  const int64_t tiles = static_cast<int64_t>(meta->total_scale_blocks) * heads;
  if (tiles > INT32_MAX) return fail(LPFA_ERR_INVALID_ARG, "too many (block, head) tiles");
  lpfa::DequantParams p;
  p.payload = payload;
  p.scales = scales;
  p.cu_seqlens = meta->dev;
  p.scale_off = meta->dev + meta->num_seqs + 1;
  p.num_seqs = meta->num_seqs;
  p.heads = heads;
  p.out = out;
  lpfa::dequantize_mxfp8_kernel<<<static_cast<unsigned>(tiles), lpfa::kDequantThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "dequantize launch");
  return LPFA_OK;
}

extern "C++" {
// Every PV mode runs over pairs of query tiles (attn_fwd_pp.cuh).
template <int kPv, bool kPerUnit>
static lpfa_status launch_attn_pp(int grid, cudaStream_t s, const CUtensorMap& tq, const CUtensorMap& tk,
                                  const CUtensorMap& tv, const lpfa::AttnParams& p) {
  constexpr uint32_t smem = lpfa::pp::smem_bytes<kPv>();
  const void* fn = reinterpret_cast<const void*>(lpfa::pp::attn_fwd_pp_kernel<kPv, kPerUnit>);
  const lpfa_status st = check_attn_kernel(fn, smem);
  if (st != LPFA_OK) return st;
  lpfa::pp::attn_fwd_pp_kernel<kPv, kPerUnit><<<grid, lpfa::kAttnThreads, smem, s>>>(tq, tk, tv, p);
  return LPFA_OK;
}
}  // extern "C++"

// Internal entry shared with the test hook: debug_stall > 0 forces a bounded wait to run out.
static lpfa_status attn_fwd_impl(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k, const uint8_t* k_sf,
                                 const uint8_t* v, const uint8_t* v_sf, const lpfa_varlen_meta* meta_q,
                                 const lpfa_varlen_meta* meta_k, int32_t heads, int32_t head_dim,
                                 lpfa_pv_mode pv_mode, const lpfa_descale* q_descale,
                                 const lpfa_descale* k_descale, const lpfa_descale* v_descale, void* out_bf16,
                                 float* lse, void* stream, int debug_stall, int shared_q = 0,
                                 bool with_ws = false, void* workspace = nullptr, size_t ws_bytes = 0) {
  if (!q || !q_sf || !k || !k_sf || !v || !out_bf16 || !lse) return fail(LPFA_ERR_INVALID_ARG, "NULL tensor pointer");
  if (pv_mode != LPFA_PV_BF16 && pv_mode != LPFA_PV_FP8 && pv_mode != LPFA_PV_BF16_V && pv_mode != LPFA_PV_MXFP8)
    return fail(LPFA_ERR_INVALID_ARG, "invalid pv_mode %d", pv_mode);
  if (pv_mode == LPFA_PV_FP8 && v_sf) return fail(LPFA_ERR_INVALID_ARG, "fp8 PV mode takes no V scale factors (v_sf must be NULL)");
  if (pv_mode == LPFA_PV_BF16_V && v_sf) return fail(LPFA_ERR_INVALID_ARG, "BF16 V input takes no V scale factors (v_sf must be NULL)");
  if (pv_mode == LPFA_PV_BF16 && !v_sf) return fail(LPFA_ERR_INVALID_ARG, "bf16 PV mode needs the V scale factors (v_sf)");
  if (pv_mode == LPFA_PV_MXFP8 && !v_sf)
    return fail(LPFA_ERR_INVALID_ARG, "MXFP8 PV mode needs V's token-orientation scale factors (v_sf)");
  if (head_dim != 128) return fail(LPFA_ERR_INVALID_ARG, "head_dim must be 128 (got %d)", head_dim);
  if (heads < 1) return fail(LPFA_ERR_INVALID_ARG, "heads must be >= 1");
  for (const lpfa_descale* d : {q_descale, k_descale, v_descale})
    if (d && d->ptr && (d->seq_stride < 0 || d->head_stride < 0))
      return fail(LPFA_ERR_INVALID_ARG, "descale strides must be >= 0");
  lpfa_status st;
  if ((st = check_meta(meta_q, "meta_q")) != LPFA_OK) return st;
  if ((st = check_meta(meta_k, "meta_k")) != LPFA_OK) return st;
  if (shared_q) {
    if (meta_q->num_seqs != 1)
      return fail(LPFA_ERR_INVALID_ARG, "a shared query set is one sequence (meta_q has %d)", meta_q->num_seqs);
  } else if (meta_q->num_seqs != meta_k->num_seqs) {
    return fail(LPFA_ERR_INVALID_ARG, "meta_q has %d sequences but meta_k has %d", meta_q->num_seqs, meta_k->num_seqs);
  }
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_sf) || !aligned16(k_sf) ||
      (v_sf && !aligned16(v_sf)) || !aligned16(out_bf16) || !aligned16(lse))
    return fail(LPFA_ERR_INVALID_ARG, "all tensors must be 16-byte aligned");
  // Output rows: the query tokens, or (shared query set) one block of them per K/V sequence.
  const int64_t out_rows = shared_q ? static_cast<int64_t>(meta_k->num_seqs) * meta_q->total_tokens
                                    : static_cast<int64_t>(meta_q->total_tokens);
  const int64_t units = shared_q ? static_cast<int64_t>(meta_k->num_seqs) * heads * ((meta_q->total_scale_blocks + 1) / 2)
                                 : static_cast<int64_t>(heads) * meta_q->total_scale_blocks;
  if (units > INT32_MAX || out_rows * heads * 128 > INT64_MAX / 4 || out_rows > INT32_MAX)
    return fail(LPFA_ERR_INVALID_ARG, "too many query tiles or output rows");
  // bf16 PV over a workspace: V is dequantized once into it, then read as BF16 V input.
  const bool dequant_v = with_ws && pv_mode == LPFA_PV_BF16;
  if (dequant_v) {
    const size_t need = static_cast<size_t>(meta_k->total_tokens) * static_cast<size_t>(heads) * 256u;
    if (!workspace) return fail(LPFA_ERR_INVALID_ARG, "bf16 PV mode needs a workspace of %zu bytes", need);
    if (!aligned16(workspace)) return fail(LPFA_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
    if (ws_bytes < need)
      return fail(LPFA_ERR_INVALID_ARG, "workspace of %zu bytes is too small (bf16 PV mode needs %zu)", ws_bytes,
                  need);
  }
  DeviceInfo info;
  if ((st = require_sm100(&info)) != LPFA_OK) return st;

  CUtensorMap tq, tk, tv;
  if ((st = payload_tmap(&tq, q, meta_q->total_tokens, heads, lpfa::kTileM)) != LPFA_OK) return st;
  if ((st = payload_tmap(&tk, k, meta_k->total_tokens, heads, lpfa::kTileN)) != LPFA_OK) return st;
  if (pv_mode == LPFA_PV_BF16_V || dequant_v) {
    // BF16 V, contiguous (Tk, H, 128): boxes of 64 elements (128 bytes) x 128 keys, 128-byte swizzle.
    if ((st = bf16_v_tmap(&tv, dequant_v ? workspace : v, meta_k->total_tokens, heads)) != LPFA_OK) return st;
  } else if ((st = payload_tmap(&tv, v, meta_k->total_tokens, heads, lpfa::kTileN)) != LPFA_OK) {
    return st;
  }

  lpfa::AttnParams p;
  p.q_sf = q_sf;
  p.k_sf = k_sf;
  p.v_sf = v_sf;
  p.cu_q = meta_q->dev;
  p.so_q = meta_q->dev + meta_q->num_seqs + 1;
  p.cu_k = meta_k->dev;
  p.so_k = meta_k->dev + meta_k->num_seqs + 1;
  // A missing descale reads the library's device constant 1.0f with zero strides.
  void* one_addr = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&one_addr, lpfa::g_lpfa_one);
  const float* one = static_cast<const float*>(one_addr);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(g_lpfa_one)");
  auto descale = [one](const lpfa_descale* d) {
    lpfa::Descale r{one, 0, 0};
    if (d && d->ptr) r = lpfa::Descale{d->ptr, d->seq_stride, d->head_stride};
    return r;
  };
  p.q_descale = descale(q_descale);
  p.k_descale = descale(k_descale);
  p.v_descale = descale(v_descale);
  p.out = static_cast<__nv_bfloat16*>(out_bf16);
  p.lse = lse;
  p.num_seqs = meta_k->num_seqs;
  p.heads = heads;
  p.tq = static_cast<int>(out_rows);
  p.total_q_tiles = meta_q->total_scale_blocks;
  p.num_units = static_cast<int>(units);
  p.debug_stall = debug_stall;
  p.shared_q = shared_q ? 1 : 0;

  const int grid = static_cast<int>(units < info.sms ? units : info.sms);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool per_unit = (p.q_descale.seq_stride | p.q_descale.head_stride | p.k_descale.seq_stride |
                         p.k_descale.head_stride) != 0;
  if (dequant_v) {
    if ((st = launch_dequant(v, v_sf, meta_k, heads, static_cast<__nv_bfloat16*>(workspace), s)) != LPFA_OK)
      return st;
    p.v_sf = nullptr;
  }
  if (pv_mode == LPFA_PV_FP8) {
    st = per_unit ? launch_attn_pp<lpfa::kPvFp8, true>(grid, s, tq, tk, tv, p)
                  : launch_attn_pp<lpfa::kPvFp8, false>(grid, s, tq, tk, tv, p);
  } else if (pv_mode == LPFA_PV_BF16 && !dequant_v) {
    st = per_unit ? launch_attn_pp<lpfa::kPvBf16Mx, true>(grid, s, tq, tk, tv, p)
                  : launch_attn_pp<lpfa::kPvBf16Mx, false>(grid, s, tq, tk, tv, p);
  } else if (pv_mode == LPFA_PV_MXFP8) {
    st = per_unit ? launch_attn_pp<lpfa::kPvMx, true>(grid, s, tq, tk, tv, p)
                  : launch_attn_pp<lpfa::kPvMx, false>(grid, s, tq, tk, tv, p);
  } else {
    st = per_unit ? launch_attn_pp<lpfa::kPvBf16In, true>(grid, s, tq, tk, tv, p)
                  : launch_attn_pp<lpfa::kPvBf16In, false>(grid, s, tq, tk, tv, p);
  }
  if (st != LPFA_OK) return st;
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  return LPFA_OK;
}

lpfa_status lpfa_attn_fwd_varlen(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k, const uint8_t* k_sf,
                                 const uint8_t* v, const uint8_t* v_sf, const lpfa_varlen_meta* meta_q,
                                 const lpfa_varlen_meta* meta_k, int32_t heads, int32_t head_dim,
                                 lpfa_pv_mode pv_mode, const float* q_descale, const float* k_descale,
                                 const float* v_descale, void* out_bf16, float* lse, void* stream) {
  const lpfa_descale qd{q_descale, 0, 0}, kd{k_descale, 0, 0}, vd{v_descale, 0, 0};
  return attn_fwd_impl(q, q_sf, k, k_sf, v, v_sf, meta_q, meta_k, heads, head_dim, pv_mode, &qd, &kd, &vd,
                       out_bf16, lse, stream, 0);
}

lpfa_status lpfa_attn_fwd_varlen_descaled(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k,
                                          const uint8_t* k_sf, const uint8_t* v, const uint8_t* v_sf,
                                          const lpfa_varlen_meta* meta_q, const lpfa_varlen_meta* meta_k,
                                          int32_t heads, int32_t head_dim, lpfa_pv_mode pv_mode,
                                          const lpfa_descale* q_descale, const lpfa_descale* k_descale,
                                          const lpfa_descale* v_descale, void* out_bf16, float* lse,
                                          void* stream) {
  return attn_fwd_impl(q, q_sf, k, k_sf, v, v_sf, meta_q, meta_k, heads, head_dim, pv_mode, q_descale, k_descale,
                       v_descale, out_bf16, lse, stream, 0);
}

}  // extern "C"

// Internal entry shared with the test hook: debug_stall > 0 forces a bounded wait to run out.
static lpfa_status attn_bwd_impl(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k, const uint8_t* k_sf,
                                 const uint8_t* v, const uint8_t* v_sf, const void* out_bf16, const void* dout_bf16,
                                 const float* lse, const lpfa_varlen_meta* meta_q, const lpfa_varlen_meta* meta_k,
                                 int32_t heads, int32_t head_dim, const lpfa_descale* q_descale,
                                 const lpfa_descale* k_descale, const lpfa_descale* v_descale, void* dq_bf16,
                                 void* dk, void* dv, uint8_t* dk_sf, uint8_t* dv_sf, int32_t output_mxfp8_dkv,
                                 void* stream, int debug_stall) {
  if (!q || !q_sf || !k || !k_sf || !v || !v_sf || !out_bf16 || !dout_bf16 || !lse || !dq_bf16 || !dk || !dv)
    return fail(LPFA_ERR_INVALID_ARG, "NULL tensor pointer");
  if (output_mxfp8_dkv != 0 && output_mxfp8_dkv != 1) return fail(LPFA_ERR_INVALID_ARG, "output_mxfp8_dkv must be 0 or 1");
  if (output_mxfp8_dkv && (!dk_sf || !dv_sf)) return fail(LPFA_ERR_INVALID_ARG, "MXFP8 dK/dV need dk_sf and dv_sf");
  if (head_dim != 128) return fail(LPFA_ERR_INVALID_ARG, "head_dim must be 128 (got %d)", head_dim);
  if (heads < 1) return fail(LPFA_ERR_INVALID_ARG, "heads must be >= 1");
  for (const lpfa_descale* d : {q_descale, k_descale, v_descale})
    if (d && d->ptr && (d->seq_stride < 0 || d->head_stride < 0))
      return fail(LPFA_ERR_INVALID_ARG, "descale strides must be >= 0");
  lpfa_status st;
  if ((st = check_meta(meta_q, "meta_q")) != LPFA_OK) return st;
  if ((st = check_meta(meta_k, "meta_k")) != LPFA_OK) return st;
  if (meta_q->num_seqs != meta_k->num_seqs)
    return fail(LPFA_ERR_INVALID_ARG, "meta_q has %d sequences but meta_k has %d", meta_q->num_seqs, meta_k->num_seqs);
  for (const void* ptr : {static_cast<const void*>(q), static_cast<const void*>(q_sf), static_cast<const void*>(k),
                          static_cast<const void*>(k_sf), static_cast<const void*>(v), static_cast<const void*>(v_sf),
                          out_bf16, dout_bf16, static_cast<const void*>(lse), static_cast<const void*>(dq_bf16),
                          static_cast<const void*>(dk), static_cast<const void*>(dv)})
    if (!aligned16(ptr)) return fail(LPFA_ERR_INVALID_ARG, "all tensors must be 16-byte aligned");
  if (output_mxfp8_dkv && (!aligned16(dk_sf) || !aligned16(dv_sf)))
    return fail(LPFA_ERR_INVALID_ARG, "all tensors must be 16-byte aligned");
  const int64_t ku = static_cast<int64_t>(heads) * meta_k->total_scale_blocks;
  const int64_t qu = static_cast<int64_t>(heads) * meta_q->total_scale_blocks;
  if (ku > INT32_MAX || qu > INT32_MAX) return fail(LPFA_ERR_INVALID_ARG, "too many tiles");
  DeviceInfo info;
  if ((st = require_sm100(&info)) != LPFA_OK) return st;
  void* one_addr = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&one_addr, lpfa::g_lpfa_one);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(g_lpfa_one)");
  const float* one = static_cast<const float*>(one_addr);
  auto descale = [one](const lpfa_descale* d) {
    lpfa::Descale r{one, 0, 0};
    if (d && d->ptr) r = lpfa::Descale{d->ptr, d->seq_stride, d->head_stride};
    return r;
  };
  lpfa::BwdParams p;
  p.q = q; p.q_sf = q_sf; p.k = k; p.k_sf = k_sf; p.v = v; p.v_sf = v_sf;
  p.o = static_cast<const __nv_bfloat16*>(out_bf16);
  p.dout = static_cast<const __nv_bfloat16*>(dout_bf16);
  p.lse = lse;
  p.cu_q = meta_q->dev;
  p.so_q = meta_q->dev + meta_q->num_seqs + 1;
  p.cu_k = meta_k->dev;
  p.so_k = meta_k->dev + meta_k->num_seqs + 1;
  p.q_descale = descale(q_descale);
  p.k_descale = descale(k_descale);
  p.v_descale = descale(v_descale);
  p.dq = static_cast<__nv_bfloat16*>(dq_bf16);
  p.dk = dk;
  p.dv = dv;
  p.dk_sf = dk_sf;
  p.dv_sf = dv_sf;
  p.num_seqs = meta_q->num_seqs;
  p.heads = heads;
  p.tq = meta_q->total_tokens;
  p.total_q_tiles = meta_q->total_scale_blocks;
  p.total_k_tiles = meta_k->total_scale_blocks;
  p.mxfp8_dkv = output_mxfp8_dkv;
  p.debug_stall = debug_stall;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (const void* fn : {reinterpret_cast<const void*>(lpfa::attn_bwd_dkdv_kernel),
                         reinterpret_cast<const void*>(lpfa::attn_bwd_dq_kernel)}) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lpfa::kBwdSmem));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  }
  if (ku > 0) {
    // D into the dQ buffer first (read by the dK/dV kernel; the dQ kernel then overwrites it).
    const int64_t rows = static_cast<int64_t>(meta_q->total_tokens) * heads;
    const int64_t blocks = std::min<int64_t>((rows + 15) / 16, static_cast<int64_t>(info.sms) * 16);
    if (blocks > 0) lpfa::attn_bwd_d_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(p);
    lpfa::attn_bwd_dkdv_kernel<<<static_cast<unsigned>(ku), lpfa::kBwdThreads, lpfa::kBwdSmem, s>>>(p);
  }
  if (qu > 0) lpfa::attn_bwd_dq_kernel<<<static_cast<unsigned>(qu), lpfa::kBwdThreads, lpfa::kBwdSmem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "backward launch");
  return LPFA_OK;
}

extern "C" {

lpfa_status lpfa_attn_fwd_shared_q(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k, const uint8_t* k_sf,
                                   const uint8_t* v, const uint8_t* v_sf, const lpfa_varlen_meta* meta_q,
                                   const lpfa_varlen_meta* meta_k, int32_t heads, int32_t head_dim,
                                   lpfa_pv_mode pv_mode, const lpfa_descale* q_descale, const lpfa_descale* k_descale,
                                   const lpfa_descale* v_descale, void* out_bf16, float* lse, void* stream) {
  return attn_fwd_impl(q, q_sf, k, k_sf, v, v_sf, meta_q, meta_k, heads, head_dim, pv_mode, q_descale, k_descale,
                       v_descale, out_bf16, lse, stream, 0, 1);
}

size_t lpfa_attn_fwd_workspace_bytes(const lpfa_varlen_meta* meta_k, int32_t heads, lpfa_pv_mode pv_mode) {
  if (!meta_k || heads < 1 || meta_k->total_tokens < 1 || pv_mode != LPFA_PV_BF16) return 0;
  return static_cast<size_t>(meta_k->total_tokens) * static_cast<size_t>(heads) * 256u;
}

lpfa_status lpfa_attn_fwd_varlen_ws(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k, const uint8_t* k_sf,
                                    const uint8_t* v, const uint8_t* v_sf, const lpfa_varlen_meta* meta_q,
                                    const lpfa_varlen_meta* meta_k, int32_t heads, int32_t head_dim,
                                    lpfa_pv_mode pv_mode, const lpfa_descale* q_descale,
                                    const lpfa_descale* k_descale, const lpfa_descale* v_descale, void* out_bf16,
                                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return attn_fwd_impl(q, q_sf, k, k_sf, v, v_sf, meta_q, meta_k, heads, head_dim, pv_mode, q_descale, k_descale,
                       v_descale, out_bf16, lse, stream, 0, 0, true, workspace, workspace_bytes);
}

lpfa_status lpfa_attn_fwd_shared_q_ws(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k,
                                      const uint8_t* k_sf, const uint8_t* v, const uint8_t* v_sf,
                                      const lpfa_varlen_meta* meta_q, const lpfa_varlen_meta* meta_k, int32_t heads,
                                      int32_t head_dim, lpfa_pv_mode pv_mode, const lpfa_descale* q_descale,
                                      const lpfa_descale* k_descale, const lpfa_descale* v_descale, void* out_bf16,
                                      float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return attn_fwd_impl(q, q_sf, k, k_sf, v, v_sf, meta_q, meta_k, heads, head_dim, pv_mode, q_descale, k_descale,
                       v_descale, out_bf16, lse, stream, 0, 1, true, workspace, workspace_bytes);
}

lpfa_status lpfa_dequantize_mxfp8_varlen(const uint8_t* payload, const uint8_t* scales, const lpfa_varlen_meta* meta,
                                         int32_t heads, int32_t head_dim, void* out_bf16, void* stream) {
  if (!payload || !scales || !out_bf16) return fail(LPFA_ERR_INVALID_ARG, "NULL tensor pointer");
  if (head_dim != 128) return fail(LPFA_ERR_INVALID_ARG, "head_dim must be 128 (got %d)", head_dim);
  if (heads < 1) return fail(LPFA_ERR_INVALID_ARG, "heads must be >= 1");
  lpfa_status st;
  if ((st = check_meta(meta, "meta")) != LPFA_OK) return st;
  if (!aligned16(payload) || !aligned16(out_bf16))
    return fail(LPFA_ERR_INVALID_ARG, "payload and out must be 16-byte aligned");
  DeviceInfo info;
  if ((st = require_sm100(&info)) != LPFA_OK) return st;
  return launch_dequant(payload, scales, meta, heads, static_cast<__nv_bfloat16*>(out_bf16),
                        static_cast<cudaStream_t>(stream));
}

lpfa_status lpfa_attn_bwd_varlen(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k, const uint8_t* k_sf,
                                 const uint8_t* v, const uint8_t* v_sf, const void* out_bf16, const void* dout_bf16,
                                 const float* lse, const lpfa_varlen_meta* meta_q, const lpfa_varlen_meta* meta_k,
                                 int32_t heads, int32_t head_dim, const lpfa_descale* q_descale,
                                 const lpfa_descale* k_descale, const lpfa_descale* v_descale, void* dq_bf16,
                                 void* dk, void* dv, uint8_t* dk_sf, uint8_t* dv_sf, int32_t output_mxfp8_dkv,
                                 void* stream) {
  return attn_bwd_impl(q, q_sf, k, k_sf, v, v_sf, out_bf16, dout_bf16, lse, meta_q, meta_k, heads, head_dim,
                       q_descale, k_descale, v_descale, dq_bf16, dk, dv, dk_sf, dv_sf, output_mxfp8_dkv, stream, 0);
}

lpfa_status lpfa_attn_bwd_varlen_debug(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k, const uint8_t* k_sf,
                                       const uint8_t* v, const uint8_t* v_sf, const void* out_bf16,
                                       const void* dout_bf16, const float* lse, const lpfa_varlen_meta* meta_q,
                                       const lpfa_varlen_meta* meta_k, int32_t heads, int32_t head_dim,
                                       const lpfa_descale* q_descale, const lpfa_descale* k_descale,
                                       const lpfa_descale* v_descale, void* dq_bf16, void* dk, void* dv,
                                       uint8_t* dk_sf, uint8_t* dv_sf, int32_t output_mxfp8_dkv, void* stream,
                                       int32_t debug_flags) {
  if (debug_flags & ~1) return fail(LPFA_ERR_INVALID_ARG, "unknown debug flags 0x%x", debug_flags);
  return attn_bwd_impl(q, q_sf, k, k_sf, v, v_sf, out_bf16, dout_bf16, lse, meta_q, meta_k, heads, head_dim,
                       q_descale, k_descale, v_descale, dq_bf16, dk, dv, dk_sf, dv_sf, output_mxfp8_dkv, stream,
                       debug_flags & 1);
}

lpfa_status lpfa_attn_fwd_varlen_debug(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k, const uint8_t* k_sf,
                                       const uint8_t* v, const uint8_t* v_sf, const lpfa_varlen_meta* meta_q,
                                       const lpfa_varlen_meta* meta_k, int32_t heads, int32_t head_dim,
                                       lpfa_pv_mode pv_mode, const float* q_descale, const float* k_descale,
                                       const float* v_descale, void* out_bf16, float* lse, void* stream,
                                       int32_t debug_flags) {
  if (debug_flags & ~1) return fail(LPFA_ERR_INVALID_ARG, "unknown debug flags 0x%x", debug_flags);
  const lpfa_descale qd{q_descale, 0, 0}, kd{k_descale, 0, 0}, vd{v_descale, 0, 0};
  return attn_fwd_impl(q, q_sf, k, k_sf, v, v_sf, meta_q, meta_k, heads, head_dim, pv_mode, &qd, &kd, &vd,
                       out_bf16, lse, stream, debug_flags & 1);
}

// ------------------------------------------------------------------ forward without allocation
// bf16 PV needs a BF16 copy of V as scratch. Callers that cannot hand the library device memory get
// it from this file-scope array instead; every GPU that loads the library holds it until exit.
static __device__ __align__(256) uint8_t g_noalloc_scratch[LPFA_NOALLOC_SCRATCH_BYTES];

namespace {
void* g_noalloc_ptr[kMaxDevices] = {};
std::mutex g_noalloc_mu;

// The scratch array's device address on the current device. In host code the array's name is only
// a host-side stand-in, so the address is looked up once per device (with it current) and kept.
lpfa_status noalloc_scratch(void** out) {
  DeviceInfo info;
  int dev = 0;
  lpfa_status st = current_device(&info, &dev);
  if (st != LPFA_OK) return st;
  std::lock_guard<std::mutex> lk(g_noalloc_mu);
  if (!g_noalloc_ptr[dev]) {
    void* ptr = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&ptr, g_noalloc_scratch);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(no-allocation scratch)");
    g_noalloc_ptr[dev] = ptr;
  }
  *out = g_noalloc_ptr[dev];
  return LPFA_OK;
}
}  // namespace

lpfa_status lpfa_attn_fwd_varlen_noalloc(const uint8_t* q, const uint8_t* q_sf, const uint8_t* k,
                                         const uint8_t* k_sf, const uint8_t* v, const uint8_t* v_sf,
                                         const lpfa_varlen_meta* meta_q, const lpfa_varlen_meta* meta_k,
                                         int32_t heads, int32_t head_dim, lpfa_pv_mode pv_mode,
                                         const lpfa_descale* q_descale, const lpfa_descale* k_descale,
                                         const lpfa_descale* v_descale, void* out_bf16, float* lse, void* stream) {
  const size_t need = lpfa_attn_fwd_workspace_bytes(meta_k, heads, pv_mode);
  if (need > static_cast<size_t>(LPFA_NOALLOC_SCRATCH_BYTES))
    return fail(LPFA_ERR_INVALID_ARG,
                "lpfa_attn_fwd_varlen_noalloc: bf16 PV over %d key tokens x %d heads needs %zu bytes of scratch; "
                "its fixed scratch holds %zu (key tokens x heads <= %zu)",
                meta_k->total_tokens, heads, need, static_cast<size_t>(LPFA_NOALLOC_SCRATCH_BYTES),
                static_cast<size_t>(LPFA_NOALLOC_SCRATCH_BYTES) / 256u);
  void* scratch = nullptr;
  if (need > 0) {
    const lpfa_status st = noalloc_scratch(&scratch);
    if (st != LPFA_OK) return st;
  }
  return attn_fwd_impl(q, q_sf, k, k_sf, v, v_sf, meta_q, meta_k, heads, head_dim, pv_mode, q_descale, k_descale,
                       v_descale, out_bf16, lse, stream, 0, 0, true, scratch, static_cast<size_t>(LPFA_NOALLOC_SCRATCH_BYTES));
}

// ---------------------------------------------------------------------------------------
// Norm and rotation of Q and K
// ---------------------------------------------------------------------------------------
namespace {

constexpr int kMaxRopeHeads = 1024;

bool rows_aligned(const lpfa_rows* r, lpfa_in_dtype dt) {
  const int vec = dt == LPFA_IN_BF16 ? 8 : 4;
  return aligned16(r->ptr) && r->tok_stride % vec == 0 && r->head_stride % vec == 0;
}

// An input (or output) of `name`, with `heads` heads where that is not 0.
lpfa_status check_rows(const lpfa_rows* r, const char* name, lpfa_in_dtype dt, int heads) {
  if (!r || !r->ptr) return fail(LPFA_ERR_INVALID_ARG, "%s is NULL", name);
  if (r->heads < 1) return fail(LPFA_ERR_INVALID_ARG, "%s has %d heads", name, r->heads);
  if (heads && r->heads != heads)
    return fail(LPFA_ERR_INVALID_ARG, "%s has %d heads, expected %d", name, r->heads, heads);
  if (!rows_aligned(r, dt))
    return fail(LPFA_ERR_INVALID_ARG, "%s must be 16-byte aligned with strides multiple of %d elements", name,
                dt == LPFA_IN_BF16 ? 8 : 4);
  return LPFA_OK;
}

// Validates what the three entry points share and fills the parameters and the plan. k may be absent.
lpfa_status rope_setup(const lpfa_rows* q, const lpfa_rows* k, lpfa_in_dtype dt, int64_t tokens, int32_t head_dim,
                       const lpfa_norm_rope* op, lpfa::RopeParams* p, lpfa::RopePlan* plan) {
  if (dt != LPFA_IN_BF16 && dt != LPFA_IN_FP32) return fail(LPFA_ERR_INVALID_ARG, "invalid input dtype %d", dt);
  if (head_dim != 128) return fail(LPFA_ERR_INVALID_ARG, "head_dim must be 128 (got %d)", head_dim);
  if (tokens < 1 || tokens > INT32_MAX) return fail(LPFA_ERR_INVALID_ARG, "tokens must be in [1, 2^31)");
  if (!op) return fail(LPFA_ERR_INVALID_ARG, "the norm and rotation (op) is NULL");
  const bool has_k = k && k->heads != 0;
  lpfa_status st;
  if ((st = check_rows(q, "q", dt, 0)) != LPFA_OK) return st;
  if (has_k && (st = check_rows(k, "k", dt, 0)) != LPFA_OK) return st;
  if (static_cast<int64_t>(q->heads) + (has_k ? k->heads : 0) > kMaxRopeHeads)
    return fail(LPFA_ERR_INVALID_ARG, "more than %d heads", kMaxRopeHeads);
  if (op->norm != 0 && op->norm != 1) return fail(LPFA_ERR_INVALID_ARG, "norm must be 0 or 1");
  if (op->norm && !(op->eps >= 0.f && std::isfinite(op->eps)))
    return fail(LPFA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (op->q_weight || op->k_weight) {
    if (op->weight_dtype != LPFA_IN_BF16 && op->weight_dtype != LPFA_IN_FP32)
      return fail(LPFA_ERR_INVALID_ARG, "invalid weight dtype %d", op->weight_dtype);
    const int vec = op->weight_dtype == LPFA_IN_BF16 ? 8 : 4;
    if (!aligned16(op->q_weight) || !aligned16(op->k_weight) || op->q_weight_head_stride % vec ||
        op->k_weight_head_stride % vec)
      return fail(LPFA_ERR_INVALID_ARG, "weights must be 16-byte aligned with strides multiple of %d elements", vec);
  }
  *p = lpfa::RopeParams{};
  *plan = lpfa::RopePlan{};
  if (op->rotary) {
    const lpfa_rotary* r = op->rotary;
    if (r->axes < 1 || r->axes > 8) return fail(LPFA_ERR_INVALID_ARG, "a rotation has 1 to 8 axes (got %d)", r->axes);
    if (r->pairing != LPFA_PAIR_INTERLEAVED && r->pairing != LPFA_PAIR_HALF)
      return fail(LPFA_ERR_INVALID_ARG, "invalid pairing %d", r->pairing);
    if (!op->positions) return fail(LPFA_ERR_INVALID_ARG, "positions is NULL");
    if (reinterpret_cast<uintptr_t>(op->positions) % (op->pos_int64 ? 8 : 4))
      return fail(LPFA_ERR_INVALID_ARG, "positions are not aligned to their type");
    for (int i = 0; i < 64; ++i) {
      if (!std::isfinite(r->inv_freq[i])) return fail(LPFA_ERR_INVALID_ARG, "frequency %d is not finite", i);
      if (r->axis[i] >= r->axes) return fail(LPFA_ERR_INVALID_ARG, "pair %d is on axis %d of %d", i, r->axis[i], r->axes);
      plan->turns[i] = r->inv_freq[i] / 6.283185307179586476925;
      plan->axis[i] = r->axis[i];
    }
    p->pos = op->positions;
    p->pos_tok = op->pos_tok_stride;
    p->pos_axis = op->pos_axis_stride;
    p->pos64 = op->pos_int64 ? 1 : 0;
  }
  p->tokens = tokens;
  p->norm = op->norm;
  p->eps = op->eps;
  p->w_bf16 = op->weight_dtype == LPFA_IN_BF16 ? 1 : 0;
  const lpfa_rows* in[2] = {q, has_k ? k : nullptr};
  for (int i = 0; i < 2; ++i) {
    if (!in[i]) continue;
    lpfa::RopeTensor& t = p->t[i];
    t.x = in[i]->ptr;
    t.tok_stride = in[i]->tok_stride;
    t.head_stride = in[i]->head_stride;
    t.heads = in[i]->heads;
    t.w = i ? op->k_weight : op->q_weight;
    t.w_head = t.w && t.heads > 1 ? (i ? op->k_weight_head_stride : op->q_weight_head_stride) : 0;
  }
  return LPFA_OK;
}

// Whether a warp's four rows are heads of one token (contiguous reads), or one head of four tokens:
// the former where every head then has its place.
int rope_quad(const lpfa::RopeParams& p) { return p.t[0].heads % 4 == 0 && p.t[1].heads % 4 == 0; }

// The forward kernel's items of work for `tiles` tiles, and its grid: two blocks per SM walk the items. All
// heads of a token share its angles, so a tile is split only where blocks would stand idle.
dim3 rope_items(lpfa::RopeParams& p, int tiles, int sms) {
  const int per_step = p.quad ? 4 : 1, slots = 2 * sms;
  int batches = 0;
  for (const lpfa::RopeTensor& t : p.t) batches += (t.heads / per_step + lpfa::kRopeBatch - 1) / lpfa::kRopeBatch;
  p.whole = tiles / slots * slots;
  const int rest = tiles - p.whole;
  const int parts = rest ? std::min(batches, slots / rest) : 1;
  p.batches = (batches + parts - 1) / parts;
  p.parts = (batches + p.batches - 1) / p.batches;
  p.items = p.whole + rest * p.parts;
  return dim3(static_cast<unsigned>(std::min(p.items, slots)));
}

int rope_weight_rows(const void* w, int64_t head_stride, int heads) {
  return !w || heads < 1 ? 0 : (head_stride != 0 ? heads : 1);
}

}  // namespace

extern "C++" {
namespace {

template <typename T, int kOut, bool kHalf>
lpfa_status launch_rope_kernel(dim3 grid, int dev, const lpfa::RopeParams& p, const lpfa::RopePlan& plan, void* stream) {
  static KernelLimits limits;
  auto kernel = lpfa::qk_norm_rope_kernel<T, kOut, kHalf>;
  constexpr int smem = lpfa::rope_smem_bytes<T>();
  const lpfa_status st = set_limits(limits, reinterpret_cast<const void*>(kernel), dev, smem, false);
  if (st != LPFA_OK) return st;
  kernel<<<grid, lpfa::kRopeThreads, smem, static_cast<cudaStream_t>(stream)>>>(p, plan);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? LPFA_OK : cuda_fail(e, "norm and rotation launch");
}

template <int kOut>
lpfa_status launch_rope(bool fp32, bool half, dim3 grid, int dev, const lpfa::RopeParams& p, const lpfa::RopePlan& plan,
                        void* stream) {
  if (fp32)
    return half ? launch_rope_kernel<float, kOut, true>(grid, dev, p, plan, stream)
                : launch_rope_kernel<float, kOut, false>(grid, dev, p, plan, stream);
  return half ? launch_rope_kernel<__nv_bfloat16, kOut, true>(grid, dev, p, plan, stream)
              : launch_rope_kernel<__nv_bfloat16, kOut, false>(grid, dev, p, plan, stream);
}

}  // namespace
}  // extern "C++"

lpfa_status lpfa_qk_norm_rope(const lpfa_rows* q, const lpfa_rows* k, lpfa_in_dtype dt, int64_t tokens,
                              int32_t head_dim, const lpfa_norm_rope* op, const lpfa_rows* q_out,
                              const lpfa_rows* k_out, lpfa_in_dtype out_dt, void* stream) {
  lpfa::RopeParams p;
  lpfa::RopePlan plan;
  lpfa_status st = rope_setup(q, k, dt, tokens, head_dim, op, &p, &plan);
  if (st != LPFA_OK) return st;
  if (out_dt != LPFA_IN_BF16 && out_dt != LPFA_IN_FP32) return fail(LPFA_ERR_INVALID_ARG, "invalid output dtype %d", out_dt);
  const lpfa_rows* out[2] = {q_out, k_out};
  for (int i = 0; i < 2; ++i) {
    if (!p.t[i].heads) continue;
    if ((st = check_rows(out[i], i ? "k_out" : "q_out", out_dt, p.t[i].heads)) != LPFA_OK) return st;
    if (out[i]->ptr == p.t[i].x && (out_dt != dt || (tokens > 1 && out[i]->tok_stride != p.t[i].tok_stride) ||
                                    (p.t[i].heads > 1 && out[i]->head_stride != p.t[i].head_stride)))
      return fail(LPFA_ERR_INVALID_ARG, "an output in its input's place needs its dtype and strides");
    p.t[i].out = out[i]->ptr;
    p.t[i].out_tok = out[i]->tok_stride;
    p.t[i].out_head = out[i]->head_stride;
  }
  DeviceInfo info;
  int dev = 0;
  if ((st = require_sm100(&info, &dev)) != LPFA_OK) return st;
  p.quad = rope_quad(p);
  const int ntok = p.quad ? lpfa::kRopeWarps : lpfa::kRopeTokens;
  const dim3 grid = rope_items(p, static_cast<int>((tokens + ntok - 1) / ntok), info.sms);
  const bool half = op->rotary && op->rotary->pairing == LPFA_PAIR_HALF;
  return out_dt == LPFA_IN_BF16 ? launch_rope<lpfa::kRopeBf16>(dt == LPFA_IN_FP32, half, grid, dev, p, plan, stream)
                                : launch_rope<lpfa::kRopeF32>(dt == LPFA_IN_FP32, half, grid, dev, p, plan, stream);
}

lpfa_status lpfa_qk_norm_rope_mxfp8(const lpfa_rows* q, const lpfa_rows* k, lpfa_in_dtype dt, int32_t head_dim,
                                    const lpfa_varlen_meta* meta, const lpfa_norm_rope* op, lpfa_scaling_mode mode,
                                    uint8_t* q_payload, uint8_t* q_scales, uint8_t* k_payload, uint8_t* k_scales,
                                    void* stream) {
  lpfa_status st = check_meta(meta, "meta");
  if (st != LPFA_OK) return st;
  lpfa::RopeParams p;
  lpfa::RopePlan plan;
  if ((st = rope_setup(q, k, dt, meta->total_tokens, head_dim, op, &p, &plan)) != LPFA_OK) return st;
  if (mode != LPFA_SCALE_RCEIL && mode != LPFA_SCALE_FLOOR) return fail(LPFA_ERR_INVALID_ARG, "invalid scaling mode %d", mode);
  uint8_t* payload[2] = {q_payload, k_payload};
  uint8_t* scales[2] = {q_scales, k_scales};
  for (int i = 0; i < 2; ++i) {
    if (!p.t[i].heads) continue;
    if (!payload[i] || !scales[i]) return fail(LPFA_ERR_INVALID_ARG, "NULL payload or scales");
    if (!aligned16(payload[i]) || !aligned16(scales[i]))
      return fail(LPFA_ERR_INVALID_ARG, "payload and scales must be 16-byte aligned");
    p.t[i].out = payload[i];
    p.t[i].scales = scales[i];
  }
  p.num_seqs = meta->num_seqs;
  p.cu_seqlens = meta->dev;
  p.scale_off = meta->dev + meta->num_seqs + 1;
  p.floor_mode = mode == LPFA_SCALE_FLOOR ? 1 : 0;
  if (meta->total_scale_blocks > INT32_MAX / 32) return fail(LPFA_ERR_INVALID_ARG, "too many tiles");
  DeviceInfo info;
  int dev = 0;
  if ((st = require_sm100(&info, &dev)) != LPFA_OK) return st;
  const bool half = op->rotary && op->rotary->pairing == LPFA_PAIR_HALF;
  p.quad = rope_quad(p);
  const int ntok = p.quad ? lpfa::kRopeWarps : lpfa::kRopeTokens;
  const dim3 grid = rope_items(p, meta->total_scale_blocks * (128 / ntok), info.sms);
  return launch_rope<lpfa::kRopeMxfp8>(dt == LPFA_IN_FP32, half, grid, dev, p, plan, stream);
}

extern "C++" {
namespace {

template <typename T, bool kHalf, bool kPerHead>
lpfa_status launch_rope_bwd_kernel(int blocks, int dev, const lpfa::RopeParams& p, const lpfa::RopePlan& plan,
                                   cudaStream_t s) {
  static KernelLimits limits;
  auto kernel = kPerHead ? lpfa::qk_norm_rope_bwd_heads_kernel<T, kHalf> : lpfa::qk_norm_rope_bwd_kernel<T, kHalf>;
  constexpr int smem = lpfa::rope_bwd_smem<T>();
  const lpfa_status st = set_limits(limits, reinterpret_cast<const void*>(kernel), dev, smem, false);
  if (st != LPFA_OK) return st;
  kernel<<<blocks, lpfa::kRopeThreads, smem, s>>>(p, plan);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? LPFA_OK : cuda_fail(e, "norm and rotation backward launch");
}

// One kernel over p's tensors, and the sums of the weight gradients behind it.
template <typename T>
lpfa_status launch_rope_bwd(bool half, bool per_head, int dev, const lpfa::RopeParams& p, const lpfa::RopePlan& plan,
                            float* dwq, float* dwk, cudaStream_t s) {
  const int blocks = static_cast<int>((p.tokens + p.tile - 1) / p.tile);
  lpfa_status st;
  if (half)
    st = per_head ? launch_rope_bwd_kernel<T, true, true>(blocks, dev, p, plan, s)
                  : launch_rope_bwd_kernel<T, true, false>(blocks, dev, p, plan, s);
  else
    st = per_head ? launch_rope_bwd_kernel<T, false, true>(blocks, dev, p, plan, s)
                  : launch_rope_bwd_kernel<T, false, false>(blocks, dev, p, plan, s);
  const int rows = p.w_rows[0] + p.w_rows[1];
  if (st != LPFA_OK || rows == 0) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows), 4);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, lpfa::qk_norm_rope_dw_kernel, static_cast<const float*>(p.partials),
                                           blocks, rows, p.w_rows[0], dwq, dwk);
  return e == cudaSuccess ? LPFA_OK : cuda_fail(e, "weight gradient launch");
}

}  // namespace
}  // extern "C++"

size_t lpfa_qk_norm_rope_bwd_workspace_bytes(int32_t q_heads, int32_t k_heads, const lpfa_norm_rope* op) {
  if (!op || q_heads < 1 || k_heads < 0) return 0;
  return static_cast<size_t>(rope_weight_rows(op->q_weight, op->q_weight_head_stride, q_heads) +
                             rope_weight_rows(op->k_weight, op->k_weight_head_stride, k_heads)) *
         128u * sizeof(float) * lpfa::kRopeBwdBlocks;
}

lpfa_status lpfa_qk_norm_rope_bwd(const lpfa_rows* dq_out, const lpfa_rows* dk_out, const lpfa_rows* q,
                                  const lpfa_rows* k, lpfa_in_dtype dt, int64_t tokens, int32_t head_dim,
                                  const lpfa_norm_rope* op, const lpfa_rows* dq, const lpfa_rows* dk,
                                  float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  lpfa::RopeParams p;
  lpfa::RopePlan plan;
  lpfa_status st = rope_setup(q, k, dt, tokens, head_dim, op, &p, &plan);
  if (st != LPFA_OK) return st;
  const lpfa_rows* in[2] = {dq_out, dk_out};
  const lpfa_rows* out[2] = {dq, dk};
  float* dw[2] = {dq_weight, dk_weight};
  for (int i = 0; i < 2; ++i) {
    lpfa::RopeTensor& t = p.t[i];
    if (!t.heads) continue;
    if ((st = check_rows(in[i], i ? "dk_out" : "dq_out", dt, t.heads)) != LPFA_OK) return st;
    if ((st = check_rows(out[i], i ? "dk" : "dq", dt, t.heads)) != LPFA_OK) return st;
    if (out[i]->ptr == in[i]->ptr && ((tokens > 1 && out[i]->tok_stride != in[i]->tok_stride) ||
                                      (t.heads > 1 && out[i]->head_stride != in[i]->head_stride)))
      return fail(LPFA_ERR_INVALID_ARG, "an output in its input's place needs its strides");
    t.dy = in[i]->ptr;
    t.dy_tok = in[i]->tok_stride;
    t.dy_head = in[i]->head_stride;
    t.out = out[i]->ptr;
    t.out_tok = out[i]->tok_stride;
    t.out_head = out[i]->head_stride;
    p.w_rows[i] = rope_weight_rows(t.w, i ? op->k_weight_head_stride : op->q_weight_head_stride, t.heads);
    if (p.w_rows[i] && (!dw[i] || !aligned16(dw[i])))
      return fail(LPFA_ERR_INVALID_ARG, "%s must be a 16-byte aligned buffer", i ? "dk_weight" : "dq_weight");
  }
  const size_t need = lpfa_qk_norm_rope_bwd_workspace_bytes(q->heads, p.t[1].heads, op);
  if (need) {
    if (!workspace || !aligned16(workspace))
      return fail(LPFA_ERR_INVALID_ARG, "the workspace must be 16-byte aligned and hold %zu bytes", need);
    if (workspace_bytes < need)
      return fail(LPFA_ERR_INVALID_ARG, "workspace of %zu bytes is too small (%zu needed)", workspace_bytes, need);
  }
  DeviceInfo info;
  int dev = 0;
  if ((st = require_sm100(&info, &dev)) != LPFA_OK) return st;
  p.quad = rope_quad(p);
  p.tile = static_cast<int>((tokens + lpfa::kRopeBwdBlocks - 1) / lpfa::kRopeBwdBlocks);
  const bool half = op->rotary && op->rotary->pairing == LPFA_PAIR_HALF;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // The tensors with one weight row (or none) in one kernel, those with a row per head in another; as a
  // rule both are of one kind.
  float* partials = static_cast<float*>(workspace);
  for (int per_head = 0; per_head < 2; ++per_head) {
    lpfa::RopeParams mine = p;
    for (int i = 0; i < 2; ++i) {
      if ((p.w_rows[i] > 1) == (per_head != 0)) continue;
      mine.t[i].heads = 0;
      mine.w_rows[i] = 0;
    }
    if (mine.t[0].heads + mine.t[1].heads == 0) continue;
    mine.partials = partials;
    partials += static_cast<int64_t>(mine.w_rows[0] + mine.w_rows[1]) * 128 * lpfa::kRopeBwdBlocks;
    st = dt == LPFA_IN_FP32 ? launch_rope_bwd<float>(half, per_head != 0, dev, mine, plan, dq_weight, dk_weight, s)
                            : launch_rope_bwd<__nv_bfloat16>(half, per_head != 0, dev, mine, plan, dq_weight, dk_weight, s);
    if (st != LPFA_OK) return st;
  }
  return LPFA_OK;
}

// ---------------------------------------------------------------------------------------
// MXFP4 cache
// ---------------------------------------------------------------------------------------
namespace {

lpfa_status kv4_setup(const lpfa_kv4_cache* c, const lpfa_page_table* table, int32_t head_dim, lpfa::Kv4Cache* out) {
  if (!c || !c->k || !c->k_sf || !c->v || !c->v_sf) return fail(LPFA_ERR_INVALID_ARG, "the cache is NULL");
  if (!table || !table->ptr) return fail(LPFA_ERR_INVALID_ARG, "the page table is NULL");
  if (head_dim != 128) return fail(LPFA_ERR_INVALID_ARG, "head_dim must be 128 (got %d)", head_dim);
  if (c->num_pages < 1 || c->heads < 1 || c->heads > kMaxRopeHeads)
    return fail(LPFA_ERR_INVALID_ARG, "the cache has %d pages of %d heads", c->num_pages, c->heads);
  int shift = 4;
  while (shift < 8 && (1 << shift) != c->page_size) ++shift;
  if ((1 << shift) != c->page_size)
    return fail(LPFA_ERR_INVALID_ARG, "page_size must be 16, 32, 64, 128 or 256 (got %d)", c->page_size);
  if (!aligned16(c->k) || !aligned16(c->k_sf) || !aligned16(c->v) || !aligned16(c->v_sf))
    return fail(LPFA_ERR_INVALID_ARG, "the cache must be 16-byte aligned");
  if (table->width < 1 || (static_cast<int64_t>(table->width) << shift) > (int64_t{1} << 30))
    return fail(LPFA_ERR_INVALID_ARG, "the page table must hold 1 to 2^30 tokens per sequence");
  if (reinterpret_cast<uintptr_t>(table->ptr) % 4) return fail(LPFA_ERR_INVALID_ARG, "the page table is misaligned");
  out->payload[0] = c->k;
  out->payload[1] = c->v;
  out->scales[0] = c->k_sf;
  out->scales[1] = c->v_sf;
  out->pages = c->num_pages;
  out->heads = c->heads;
  out->page_size = c->page_size;
  out->page_shift = shift;
  out->table = table->ptr;
  out->table_stride = table->seq_stride;
  out->width = table->width;
  return LPFA_OK;
}

}  // namespace

lpfa_status lpfa_kv4_write(const lpfa_rows* k, const lpfa_rows* v, lpfa_in_dtype dt, int32_t head_dim,
                           const lpfa_kv4_cache* cache, const lpfa_page_table* table, const int32_t* start,
                           const lpfa_varlen_meta* meta, lpfa_scaling_mode mode, void* stream) {
  lpfa::Kv4WriteParams p = {};
  lpfa_status st = kv4_setup(cache, table, head_dim, &p.c);
  if (st != LPFA_OK) return st;
  if (dt != LPFA_IN_BF16 && dt != LPFA_IN_FP32) return fail(LPFA_ERR_INVALID_ARG, "invalid input dtype %d", dt);
  if (mode != LPFA_SCALE_RCEIL && mode != LPFA_SCALE_FLOOR) return fail(LPFA_ERR_INVALID_ARG, "invalid scaling mode %d", mode);
  if ((st = check_meta(meta, "meta")) != LPFA_OK) return st;
  const lpfa_rows* in[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    if ((st = check_rows(in[i], i ? "v" : "k", dt, cache->heads)) != LPFA_OK) return st;
    p.x[i] = in[i]->ptr;
    p.tok_stride[i] = in[i]->tok_stride;
    p.head_stride[i] = in[i]->head_stride;
  }
  if (reinterpret_cast<uintptr_t>(start) % 4) return fail(LPFA_ERR_INVALID_ARG, "start is misaligned");
  p.num_seqs = meta->num_seqs;
  p.cu_seqlens = meta->dev;
  p.start = start;
  p.tokens = meta->total_tokens;
  p.floor_mode = mode == LPFA_SCALE_FLOOR ? 1 : 0;
  DeviceInfo info;
  int dev = 0;
  if ((st = require_sm100(&info, &dev)) != LPFA_OK) return st;
  // One token per block while there are few, else up to 32 that share their table lookups.
  p.tile = std::min(lpfa::kKv4Tile, (p.tokens + 4 * info.sms - 1) / (4 * info.sms));
  const dim3 grid(static_cast<unsigned>((p.tokens + p.tile - 1) / p.tile), 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dt == LPFA_IN_FP32)
    lpfa::kv4_write_kernel<float><<<grid, lpfa::kKv4Threads, 0, s>>>(p);
  else
    lpfa::kv4_write_kernel<__nv_bfloat16><<<grid, lpfa::kKv4Threads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? LPFA_OK : cuda_fail(e, "cache write launch");
}

lpfa_status lpfa_kv4_read(const lpfa_kv4_cache* cache, const lpfa_page_table* table, const int32_t* start,
                          const lpfa_varlen_meta* meta, int32_t head_dim, uint8_t* k_payload, uint8_t* k_scales,
                          uint8_t* v_payload, uint8_t* v_scales, void* stream) {
  lpfa::Kv4ReadParams p = {};
  lpfa_status st = kv4_setup(cache, table, head_dim, &p.c);
  if (st != LPFA_OK) return st;
  if ((st = check_meta(meta, "meta")) != LPFA_OK) return st;
  if (!k_payload || !k_scales || !v_payload || !v_scales) return fail(LPFA_ERR_INVALID_ARG, "NULL payload or scales");
  if (!aligned16(k_payload) || !aligned16(k_scales) || !aligned16(v_payload) || !aligned16(v_scales))
    return fail(LPFA_ERR_INVALID_ARG, "payload and scales must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(start) % 4) return fail(LPFA_ERR_INVALID_ARG, "start is misaligned");
  if (meta->total_scale_blocks > INT32_MAX / 32) return fail(LPFA_ERR_INVALID_ARG, "too many tiles");
  p.payload[0] = k_payload;
  p.payload[1] = v_payload;
  p.scales[0] = k_scales;
  p.scales[1] = v_scales;
  p.num_seqs = meta->num_seqs;
  p.cu_seqlens = meta->dev;
  p.scale_off = meta->dev + meta->num_seqs + 1;
  p.start = start;
  DeviceInfo info;
  int dev = 0;
  if ((st = require_sm100(&info, &dev)) != LPFA_OK) return st;
  const dim3 grid(static_cast<unsigned>(meta->total_scale_blocks) * 4u, 2);
  // The limit is the kernel's largest need, not this call's: another thread may be about to launch with more heads.
  static KernelLimits limits;
  constexpr int kMost = kMaxRopeHeads * lpfa::kKv4Tile * 4;  // 128 KB
  st = set_limits(limits, reinterpret_cast<const void*>(lpfa::kv4_read_kernel), dev, kMost, false);
  if (st != LPFA_OK) return st;
  const int smem = cache->heads * lpfa::kKv4Tile * 4;
  lpfa::kv4_read_kernel<<<grid, lpfa::kKv4Threads, static_cast<size_t>(smem), static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? LPFA_OK : cuda_fail(e, "cache read launch");
}

extern "C++" {
namespace {

// Clusters of n blocks of the cache attention that the current device runs at a time, looked up once.
template <int kTiles>
int attn4_clusters(const cudaLaunchConfig_t& cfg, int dev, int n) {
  static int known[kMaxDevices][lpfa::kAttn4MaxSplit + 1] = {};  // 0: not looked up; else count + 1
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  int& k = known[dev][n];
  if (k == 0) {
    int count = 0;
    if (cudaOccupancyMaxActiveClusters(&count, lpfa::attn_kv4_kernel<kTiles>, &cfg) != cudaSuccess) {
      cudaGetLastError();  // a size that this device does not have
      count = 0;
    }
    k = count + 1;
  }
  return k - 1;
}

template <int kTiles>
lpfa_status launch_attn_kv4(lpfa::Attn4Params& p, int64_t max_rows, int sms, int dev, cudaStream_t s) {
  constexpr uint32_t smem = lpfa::attn4_smem_bytes<kTiles>();
  auto kernel = lpfa::attn_kv4_kernel<kTiles>;
  static KernelLimits limits;
  const lpfa_status st = set_limits(limits, reinterpret_cast<const void*>(kernel), dev, static_cast<int>(smem), true);
  if (st != LPFA_OK) return st;
  const int64_t tiles = (max_rows + 8 * kTiles - 1) / (8 * kTiles);
  const int64_t work = tiles * p.c.heads * p.num_seqs;
  if (work > INT32_MAX / lpfa::kAttn4MaxSplit) return fail(LPFA_ERR_INVALID_ARG, "too many query tiles");
  p.tiles = static_cast<int>(tiles);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(32 * lpfa::attn4_warps<kTiles>());
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // As many blocks as run at a time, two per SM, but 128 keys for each at least. (Two rounds of half
  // as long blocks take 27 instead of 16 us for 8 x 5 query tokens over up to 4096 keys.) Clusters beyond
  // the portable size of 8 only where the device can place all of them at once.
  const int64_t keys = static_cast<int64_t>(p.c.width) << p.c.page_shift;
  p.splits = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>({lpfa::kAttn4MaxSplit, 2 * sms / work, keys / 128})));
  for (;; --p.splits) {
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
    cfg.gridDim = dim3(static_cast<unsigned>(work * p.splits));
    if (p.splits <= 8 || attn4_clusters<kTiles>(cfg, dev, p.splits) >= work) break;
  }
  // Blocks that have to wait for others' places run in order of length, where there are few rounds of them and the
  // order matters more than its cost (8 key heads, with and without: 64 ragged sequences of up to 8192 keys
  // 70 and 99 us, 128 of 2000 53 and 56; 256 of 2000, 7 rounds, 100 either way, 512 of 300 110 and 92).
  p.sorted = p.num_seqs > 1 && work * p.splits > 2 * sms && work * p.splits <= 2 * sms * lpfa::kAttn4SortRounds;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess ? LPFA_OK : cuda_fail(e, "cache attention launch");
}

}  // namespace
}  // extern "C++"

lpfa_status lpfa_attn_fwd_kv4(const lpfa_rows* q, int32_t head_dim, const lpfa_kv4_cache* cache,
                              const lpfa_page_table* table, const int32_t* kv_lens, const lpfa_varlen_meta* meta_q,
                              int32_t causal, void* out_bf16, float* lse, void* stream) {
  lpfa::Attn4Params p = {};
  lpfa_status st = kv4_setup(cache, table, head_dim, &p.c);
  if (st != LPFA_OK) return st;
  if ((st = check_rows(q, "q", LPFA_IN_BF16, 0)) != LPFA_OK) return st;
  if ((st = check_meta(meta_q, "meta_q")) != LPFA_OK) return st;
  if (!kv_lens || !out_bf16 || !lse) return fail(LPFA_ERR_INVALID_ARG, "NULL tensor pointer");
  if (q->heads % cache->heads || q->heads > 65536)
    return fail(LPFA_ERR_INVALID_ARG, "%d query heads over %d cached heads: not a multiple", q->heads, cache->heads);
  if (causal != 0 && causal != 1) return fail(LPFA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!aligned16(out_bf16) || !aligned16(lse) || reinterpret_cast<uintptr_t>(kv_lens) % 4)
    return fail(LPFA_ERR_INVALID_ARG, "out and lse must be 16-byte aligned, kv_lens 4-byte aligned");
  p.q = static_cast<const __nv_bfloat16*>(q->ptr);
  p.q_tok = q->tok_stride;
  p.q_head = q->head_stride;
  p.cu_q = meta_q->dev;
  p.kv_lens = kv_lens;
  p.num_seqs = meta_q->num_seqs;
  p.heads_q = q->heads;
  p.group = q->heads / cache->heads;
  p.causal = causal;
  p.total_q = meta_q->total_tokens;
  p.out = static_cast<__nv_bfloat16*>(out_bf16);
  p.lse = lse;
  const int64_t max_rows = static_cast<int64_t>(meta_q->max_seqlen) * p.group;
  if (max_rows > INT32_MAX / 2) return fail(LPFA_ERR_INVALID_ARG, "too many query rows in a sequence");
  DeviceInfo info;
  int dev = 0;
  if ((st = require_sm100(&info, &dev)) != LPFA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // One row costs what eight do. Sixteen per block cost 5/3 as much as eight (conversions and reads of the
  // cache are shared) with half as many warps on an SM: taken where that is less work for the longest
  // sequence's rows, and where the largest split still fills the card. (16 rows over 8 key heads: 32 x 8192
  // keys 105 instead of 143 us; where the split would not fill it, 1 x 65536 58 instead of 50 and 4 x 2048
  // 14.4 instead of 12.8, though 4 x 65536 106 instead of 138; 20 rows over 4 heads of 8 x 4096 keys 19
  // instead of 17.)
  const int64_t tiles16 = (max_rows + 15) / 16, tiles8 = (max_rows + 7) / 8;
  const bool sixteen = 5 * tiles16 < 3 * tiles8 && tiles16 * p.c.heads * p.num_seqs * 8 >= 2 * info.sms;
  return sixteen ? launch_attn_kv4<2>(p, max_rows, info.sms, dev, s) : launch_attn_kv4<1>(p, max_rows, info.sms, dev, s);
}

lpfa_status lpfa_device_status(void* stream, int32_t* detail) {
  if (detail) *detail = 0;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  int32_t word[2] = {0, 0};
  e = cudaMemcpyFromSymbol(word, lpfa::g_lpfa_status, sizeof(word));
  if (e != cudaSuccess) return cuda_fail(e, "reading the device status word");
  if (word[0] != 0) {
    const int32_t zero[2] = {0, 0};
    e = cudaMemcpyToSymbol(lpfa::g_lpfa_status, zero, sizeof(zero));
    if (e != cudaSuccess) return cuda_fail(e, "resetting the device status word");
    if (detail) *detail = word[1];
    if (word[0] == LPFA_ERR_INVALID_ARG)
      return fail(LPFA_ERR_INVALID_ARG, "a length, start or page table entry in device memory is out of range (site %d)",
                  word[1]);
    return fail(LPFA_ERR_TIMEOUT, "a kernel gave up waiting on a barrier (site %d)", word[1]);
  }
  return LPFA_OK;
}

}  // extern "C"
