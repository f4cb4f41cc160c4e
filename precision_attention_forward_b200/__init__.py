"""Python binding of liblpfa: MXFP8 varlen quantization, block-scaled attention forward and backward,
the norm and rotation of Q and K before them, and a paged MXFP4 key/value cache with its attention.

Argument marshalling only: every step of the path runs in the library's CUDA kernels
(``liblpfa.so``, built in-tree for sm_100a). PyTorch provides device memory and streams.
Importing this package fails if the library has not been built; there is no CPU fallback.

Every function that takes `stream` enqueues its work there (None: the current stream) and returns without waiting.
With another stream than the current one, the caller orders it behind the work that made the inputs, and keeps the
tensors that it hands in alive, or recorded on that stream, until the work is done.

The functions carry the C ABI's names (``include/lpfa.h``); the LP-FA4 README names
(``Mxfp8VarlenMeta.from_lengths``, ``quantize_mxfp8_varlen``,
``mxfp8_flash_attn_varlen_forward``) are provided as aliases.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np
import torch

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "liblpfa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        "liblpfa.so is not built; run `python precision_attention_forward_b200/build.py` "
        "(the library has no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)

LPFA_OK, LPFA_ERR_INVALID_ARG, LPFA_ERR_UNSUPPORTED, LPFA_ERR_CUDA, LPFA_ERR_TIMEOUT = 0, 1, 2, 3, 4
_STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CUDA", 4: "TIMEOUT"}
IN_DTYPES = {"bf16": 0, "fp32": 1}
SCALING_MODES = {"rceil": 0, "floor": 1}
PV_MODES = {"bf16": 0, "fp8": 1, "bf16v": 2, "mxfp8": 3}  # bf16v: BF16 V input, bf16 PV; mxfp8: block-scaled PV

# Symbols the header declares; the tests check that each one is exported.
EXPORTED_SYMBOLS = (
    "lpfa_meta_dev_ints", "lpfa_varlen_meta_fill_host", "lpfa_varlen_meta_from_lengths",
    "lpfa_scale_bytes", "lpfa_quantize_mxfp8_varlen", "lpfa_cast_e4m3", "lpfa_attn_fwd_varlen",
    "lpfa_device_status", "lpfa_last_error_message", "lpfa_version", "lpfa_attn_fwd_varlen_debug",
    "lpfa_attn_fwd_varlen_descaled", "lpfa_quantize_mxfp8_varlen_tokens", "lpfa_attn_bwd_varlen",
    "lpfa_attn_bwd_varlen_debug", "lpfa_attn_fwd_shared_q", "lpfa_dequantize_mxfp8_varlen",
    "lpfa_attn_fwd_workspace_bytes", "lpfa_attn_fwd_varlen_ws", "lpfa_attn_fwd_shared_q_ws",
    "lpfa_attn_fwd_varlen_noalloc", "lpfa_qk_norm_rope", "lpfa_qk_norm_rope_mxfp8",
    "lpfa_qk_norm_rope_bwd_workspace_bytes", "lpfa_qk_norm_rope_bwd", "lpfa_kv4_write", "lpfa_kv4_read",
    "lpfa_attn_fwd_kv4",
)


class LpfaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"lpfa status {_STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class _Descale(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("seq_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Meta(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int32),
                ("total_scale_blocks", ctypes.c_int32), ("max_seqlen", ctypes.c_int32),
                ("dev", ctypes.c_void_p)]


class _Rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("tok_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32)]


class _Rotary(ctypes.Structure):
    _fields_ = [("axes", ctypes.c_int32), ("pairing", ctypes.c_int32), ("inv_freq", ctypes.c_double * 64),
                ("axis", ctypes.c_uint8 * 64)]


class _NormRope(ctypes.Structure):
    _fields_ = [("rotary", ctypes.POINTER(_Rotary)), ("positions", ctypes.c_void_p), ("pos_tok_stride", ctypes.c_int64),
                ("pos_axis_stride", ctypes.c_int64), ("pos_int64", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p), ("q_weight_head_stride", ctypes.c_int64),
                ("k_weight", ctypes.c_void_p), ("k_weight_head_stride", ctypes.c_int64),
                ("weight_dtype", ctypes.c_int)]


class _Kv4Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("k_sf", ctypes.c_void_p), ("v", ctypes.c_void_p), ("v_sf", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("heads", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class _PageTable(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("seq_stride", ctypes.c_int64), ("width", ctypes.c_int32)]


_vp, _i32, _i64, _f32p = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
_lib.lpfa_meta_dev_ints.argtypes = [_i32]
_lib.lpfa_meta_dev_ints.restype = ctypes.c_size_t
_lib.lpfa_varlen_meta_fill_host.argtypes = [_vp, _i32, _vp, ctypes.POINTER(_Meta)]
_lib.lpfa_varlen_meta_fill_host.restype = ctypes.c_int
_lib.lpfa_varlen_meta_from_lengths.argtypes = [_vp, _i32, ctypes.POINTER(_Meta), _vp]
_lib.lpfa_varlen_meta_from_lengths.restype = ctypes.c_int
_lib.lpfa_scale_bytes.argtypes = [ctypes.POINTER(_Meta), _i32]
_lib.lpfa_scale_bytes.restype = ctypes.c_size_t
_lib.lpfa_quantize_mxfp8_varlen.argtypes = [_vp, ctypes.c_int, _i64, _i64, _i32, _i32, ctypes.POINTER(_Meta),
                                            ctypes.c_int, _vp, _vp, _vp]
_lib.lpfa_quantize_mxfp8_varlen.restype = ctypes.c_int
_lib.lpfa_quantize_mxfp8_varlen_tokens.argtypes = _lib.lpfa_quantize_mxfp8_varlen.argtypes
_lib.lpfa_quantize_mxfp8_varlen_tokens.restype = ctypes.c_int
_lib.lpfa_attn_bwd_varlen.argtypes = ([_vp] * 9 + [ctypes.POINTER(_Meta), ctypes.POINTER(_Meta), _i32, _i32] +
                                      [ctypes.POINTER(_Descale)] * 3 + [_vp] * 5 + [_i32, _vp])
_lib.lpfa_attn_bwd_varlen.restype = ctypes.c_int
_lib.lpfa_attn_bwd_varlen_debug.argtypes = list(_lib.lpfa_attn_bwd_varlen.argtypes) + [_i32]
_lib.lpfa_attn_bwd_varlen_debug.restype = ctypes.c_int
_lib.lpfa_cast_e4m3.argtypes = [_vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp]
_lib.lpfa_cast_e4m3.restype = ctypes.c_int
_lib.lpfa_attn_fwd_varlen.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(_Meta), ctypes.POINTER(_Meta),
                                      _i32, _i32, ctypes.c_int, _f32p, _f32p, _f32p, _vp, _vp, _vp]
_lib.lpfa_attn_fwd_varlen.restype = ctypes.c_int
_lib.lpfa_attn_fwd_varlen_debug.argtypes = list(_lib.lpfa_attn_fwd_varlen.argtypes) + [_i32]
_lib.lpfa_attn_fwd_varlen_descaled.argtypes = (list(_lib.lpfa_attn_fwd_varlen.argtypes[:11]) +
                                               [ctypes.POINTER(_Descale)] * 3 + [_vp, _vp, _vp])
_lib.lpfa_attn_fwd_varlen_descaled.restype = ctypes.c_int
_lib.lpfa_attn_fwd_shared_q.argtypes = _lib.lpfa_attn_fwd_varlen_descaled.argtypes
_lib.lpfa_attn_fwd_shared_q.restype = ctypes.c_int
_lib.lpfa_attn_fwd_varlen_debug.restype = ctypes.c_int
_lib.lpfa_attn_fwd_varlen_ws.argtypes = (list(_lib.lpfa_attn_fwd_varlen_descaled.argtypes[:16]) +
                                         [_vp, ctypes.c_size_t, _vp])
_lib.lpfa_attn_fwd_varlen_ws.restype = ctypes.c_int
_lib.lpfa_attn_fwd_shared_q_ws.argtypes = _lib.lpfa_attn_fwd_varlen_ws.argtypes
_lib.lpfa_attn_fwd_shared_q_ws.restype = ctypes.c_int
_lib.lpfa_attn_fwd_varlen_noalloc.argtypes = _lib.lpfa_attn_fwd_varlen_descaled.argtypes
_lib.lpfa_attn_fwd_varlen_noalloc.restype = ctypes.c_int
_lib.lpfa_attn_fwd_workspace_bytes.argtypes = [ctypes.POINTER(_Meta), _i32, ctypes.c_int]
_lib.lpfa_attn_fwd_workspace_bytes.restype = ctypes.c_size_t
_lib.lpfa_dequantize_mxfp8_varlen.argtypes = [_vp, _vp, ctypes.POINTER(_Meta), _i32, _i32, _vp, _vp]
_lib.lpfa_dequantize_mxfp8_varlen.restype = ctypes.c_int
_rows_p, _op_p = ctypes.POINTER(_Rows), ctypes.POINTER(_NormRope)
_lib.lpfa_qk_norm_rope.argtypes = [_rows_p, _rows_p, ctypes.c_int, _i64, _i32, _op_p, _rows_p, _rows_p, ctypes.c_int,
                                   _vp]
_lib.lpfa_qk_norm_rope.restype = ctypes.c_int
_lib.lpfa_qk_norm_rope_mxfp8.argtypes = [_rows_p, _rows_p, ctypes.c_int, _i32, ctypes.POINTER(_Meta), _op_p,
                                         ctypes.c_int, _vp, _vp, _vp, _vp, _vp]
_lib.lpfa_qk_norm_rope_mxfp8.restype = ctypes.c_int
_lib.lpfa_qk_norm_rope_bwd_workspace_bytes.argtypes = [_i32, _i32, _op_p]
_lib.lpfa_qk_norm_rope_bwd_workspace_bytes.restype = ctypes.c_size_t
_lib.lpfa_qk_norm_rope_bwd.argtypes = ([_rows_p] * 4 + [ctypes.c_int, _i64, _i32, _op_p, _rows_p, _rows_p, _vp, _vp,
                                                        _vp, ctypes.c_size_t, _vp])
_lib.lpfa_qk_norm_rope_bwd.restype = ctypes.c_int
_cache_p, _table_p = ctypes.POINTER(_Kv4Cache), ctypes.POINTER(_PageTable)
_lib.lpfa_kv4_write.argtypes = [_rows_p, _rows_p, ctypes.c_int, _i32, _cache_p, _table_p, _vp, ctypes.POINTER(_Meta),
                                ctypes.c_int, _vp]
_lib.lpfa_kv4_write.restype = ctypes.c_int
_lib.lpfa_kv4_read.argtypes = [_cache_p, _table_p, _vp, ctypes.POINTER(_Meta), _i32, _vp, _vp, _vp, _vp, _vp]
_lib.lpfa_kv4_read.restype = ctypes.c_int
_lib.lpfa_attn_fwd_kv4.argtypes = [_rows_p, _i32, _cache_p, _table_p, _vp, ctypes.POINTER(_Meta), _i32, _vp, _vp, _vp]
_lib.lpfa_attn_fwd_kv4.restype = ctypes.c_int
_lib.lpfa_device_status.argtypes = [_vp, ctypes.POINTER(_i32)]
_lib.lpfa_device_status.restype = ctypes.c_int
_lib.lpfa_last_error_message.argtypes = []
_lib.lpfa_last_error_message.restype = ctypes.c_char_p
_lib.lpfa_version.argtypes = []
_lib.lpfa_version.restype = ctypes.c_char_p


def _check(status: int) -> None:
    if status != LPFA_OK:
        raise LpfaError(status, _lib.lpfa_last_error_message().decode(errors="replace"))


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def lpfa_version() -> str:
    return _lib.lpfa_version().decode()


class VarlenMeta:
    """Packed varlen metadata: host scalars plus a device int32 buffer (cu_seqlens | scale_off)."""

    def __init__(self, lengths, c_meta: _Meta, dev: Optional[torch.Tensor], host_ints: np.ndarray):
        self.lengths = np.asarray(lengths, dtype=np.int32)
        self._c = c_meta
        self.dev = dev
        self.host_ints = host_ints

    num_seqs = property(lambda self: self._c.num_seqs)
    total_tokens = property(lambda self: self._c.total_tokens)
    total_scale_blocks = property(lambda self: self._c.total_scale_blocks)
    max_seqlen = property(lambda self: self._c.max_seqlen)

    @property
    def cu_seqlens(self) -> np.ndarray:
        return self.host_ints[: self.num_seqs + 1]

    @property
    def scale_off(self) -> np.ndarray:
        return self.host_ints[self.num_seqs + 1:]

    def scale_bytes(self, heads: int) -> int:
        return int(_lib.lpfa_scale_bytes(ctypes.byref(self._c), heads))

    @classmethod
    def from_lengths(cls, lengths: Sequence[int], device="cuda", stream=None) -> "VarlenMeta":
        return lpfa_varlen_meta_from_lengths(lengths, device=device, stream=stream)


def lpfa_varlen_meta_fill_host(lengths: Sequence[int]) -> VarlenMeta:
    """Host-only metadata (no device buffer); usable without a GPU."""
    lens = np.ascontiguousarray(np.asarray(lengths, dtype=np.int32))
    n = int(lens.size)
    host = np.zeros(max(int(_lib.lpfa_meta_dev_ints(n)), 1), dtype=np.int32)
    m = _Meta()
    _check(_lib.lpfa_varlen_meta_fill_host(lens.ctypes.data if n else None, n, host.ctypes.data, ctypes.byref(m)))
    return VarlenMeta(lens, m, None, host)


def lpfa_varlen_meta_from_lengths(lengths: Sequence[int], device="cuda", stream=None) -> VarlenMeta:
    lens = np.ascontiguousarray(np.asarray(lengths, dtype=np.int32))
    n = int(lens.size)
    host_meta = lpfa_varlen_meta_fill_host(lens)
    dev = torch.empty(int(_lib.lpfa_meta_dev_ints(n)), dtype=torch.int32, device=device)
    m = _Meta()
    m.dev = dev.data_ptr()
    with torch.cuda.device(dev.device):
        _check(_lib.lpfa_varlen_meta_from_lengths(lens.ctypes.data, n, ctypes.byref(m), _stream_ptr(stream)))
    return VarlenMeta(lens, m, dev, host_meta.host_ints)


def _strides(x: torch.Tensor):
    if x.dim() != 3 or x.shape[2] != 128 or x.stride(2) != 1:
        raise ValueError("expected a (tokens, heads, 128) tensor with a contiguous last dimension")
    return x.stride(0), x.stride(1)


def lpfa_quantize_mxfp8_varlen(x: torch.Tensor, meta: VarlenMeta, scaling_mode: str = "rceil",
                               payload: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                               stream=None, orientation: str = "head_dim"):
    """Quantize packed (T, H, 128) bf16/fp32 to (payload uint8 (T,H,128), scales uint8 (blocks*H*512,)).

    orientation "head_dim": one scale per 32 elements along head_dim (Q and K, and V in bf16 PV
    mode); "tokens": one scale per 32 tokens of a channel (V in mxfp8 PV mode).
    """
    if orientation not in ("head_dim", "tokens"):
        raise ValueError("orientation must be 'head_dim' or 'tokens'")
    dt = {torch.bfloat16: "bf16", torch.float32: "fp32"}.get(x.dtype)
    if dt is None:
        raise ValueError("x must be bf16 or fp32")
    if scaling_mode not in SCALING_MODES:
        raise ValueError("scaling_mode must be 'rceil' or 'floor'")
    ts, hs = _strides(x)
    T, H = x.shape[0], x.shape[1]
    if T != meta.total_tokens:
        raise ValueError("x has %d tokens but the metadata describes %d" % (T, meta.total_tokens))
    if payload is None:
        payload = torch.empty((T, H, 128), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(meta.scale_bytes(H), dtype=torch.uint8, device=x.device)
    with torch.cuda.device(x.device):
        fn = _lib.lpfa_quantize_mxfp8_varlen if orientation == "head_dim" else _lib.lpfa_quantize_mxfp8_varlen_tokens
        _check(fn(x.data_ptr(), IN_DTYPES[dt], ts, hs, H, 128, ctypes.byref(meta._c),
                  SCALING_MODES[scaling_mode], payload.data_ptr(), scales.data_ptr(), _stream_ptr(stream)))
    return payload, scales


def lpfa_cast_e4m3(v: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Unscaled E4M3 cast of a bf16 (T, H, 128) tensor (fp8 PV mode V)."""
    if v.dtype != torch.bfloat16:
        raise ValueError("v must be bf16")
    ts, hs = _strides(v)
    T, H = v.shape[0], v.shape[1]
    if out is None:
        out = torch.empty((T, H, 128), dtype=torch.uint8, device=v.device)
    with torch.cuda.device(v.device):
        _check(_lib.lpfa_cast_e4m3(v.data_ptr(), ts, hs, T, H, 128, out.data_ptr(), _stream_ptr(stream)))
    return out


def descale_strides(t: torch.Tensor, num_seqs: int, heads: int):
    """(seq_stride, head_stride) in elements of a descale tensor indexed by (sequence, head).

    Accepted shapes (vLLM #63232: per-tensor and per-head scales keep their descale tensors;
    FA4's descale views are (batch, kv_heads)): one element (per tensor), (heads,) (per head),
    and (S, Hd) with S in {1, num_seqs}, Hd in {1, heads}; size-1 axes broadcast (stride 0).
    """
    if t.dtype != torch.float32:
        raise ValueError("a descale must be a float32 tensor")
    if t.numel() == 1:
        return 0, 0
    if t.dim() == 1 and t.shape[0] == heads:
        return 0, t.stride(0)
    if t.dim() == 2 and t.shape[0] in (1, num_seqs) and t.shape[1] in (1, heads):
        return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else 0)
    raise ValueError("a descale has one element, shape (heads,) or (num_seqs or 1, heads or 1); got %s"
                     % (tuple(t.shape),))


def _check_packed(q, q_sf, k, k_sf, v, v_sf, meta_q: "VarlenMeta", meta_k: "VarlenMeta", v_dtype) -> None:
    """Q, K and V and their scale storage hold what the kernels will read of them: one head count for all
    three, at least the metadata's tokens, and scales for their blocks. (A missing v_sf is the library's to refuse.)"""
    H = q.shape[1] if q.dim() == 3 else 0
    for name, t, meta, dtype in (("q", q, meta_q, torch.uint8), ("k", k, meta_k, torch.uint8), ("v", v, meta_k, v_dtype)):
        if (t.dtype != dtype or t.dim() != 3 or t.shape[0] < meta.total_tokens or t.shape[1] != H or t.shape[2] != 128
                or not t.is_contiguous() or t.device != q.device):
            raise ValueError("%s must be a contiguous %s (tokens, heads, 128) tensor on the device of q with the %d tokens "
                             "of its metadata and q's %d heads, not %s" % (name, dtype, meta.total_tokens, H, tuple(t.shape)))
    for name, t, meta in (("q_sf", q_sf, meta_q), ("k_sf", k_sf, meta_k), ("v_sf", v_sf, meta_k)):
        if t is None and name == "v_sf":
            continue
        if t.numel() * t.element_size() < meta.scale_bytes(H) or not t.is_contiguous() or t.device != q.device:
            raise ValueError("%s must hold %d contiguous scale bytes on the device of q" % (name, meta.scale_bytes(H)))


def _check_out_lse(out, lse, rows: int, heads: int, device) -> None:
    """Given outputs of the forward (None: allocated) hold what it writes."""
    for name, t, dtype, shape in (("out", out, torch.bfloat16, (rows, heads, 128)), ("lse", lse, torch.float32, (heads, rows))):
        if t is not None and (t.dtype != dtype or t.numel() < np.prod(shape) or not t.is_contiguous() or t.device != device):
            raise ValueError("%s must be a contiguous %s tensor of shape %s on the device of q" % (name, dtype, shape))


def lpfa_attn_fwd_varlen(q: torch.Tensor, q_sf: torch.Tensor, k: torch.Tensor, k_sf: torch.Tensor,
                         v: torch.Tensor, v_sf: Optional[torch.Tensor], meta_q: VarlenMeta, meta_k: VarlenMeta,
                         pv_mode: str = "bf16", q_descale: Optional[torch.Tensor] = None,
                         k_descale: Optional[torch.Tensor] = None, v_descale: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None,
                         debug_flags: int = 0, workspace=True):
    """Block-scaled attention forward; returns (out bf16 (Tq,H,128), lse fp32 (H,Tq)).

    Every query sees every key of its sequence; Q, K and V have the same heads.
    q/k/v_descale: None (exactly 1.0), a one-element tensor (per tensor), (H,) (per head) or
    (S, H) (per sequence and head), float32 on the device; see descale_strides.
    workspace: where the bf16 PV mode converts V to BF16 once (lpfa_attn_fwd_varlen_ws): True
    allocates it, a uint8 device tensor of at least lpfa_attn_fwd_workspace_bytes bytes is used as
    is, False converts V tiles inside the attention kernel instead (same bits). Other modes ignore it.
    (An allocated workspace is recorded on `stream` when that is a torch.cuda.Stream; with a raw
    stream handle other than the current stream, pass a workspace tensor that outlives the work.)
    debug_flags != 0 goes through lpfa_attn_fwd_varlen_debug (test hook, see include/lpfa.h),
    which takes per-tensor descales only and no workspace.
    """
    if pv_mode not in PV_MODES:
        raise ValueError("pv_mode must be 'bf16', 'fp8', 'bf16v' or 'mxfp8'")
    _check_packed(q, q_sf, k, k_sf, v, v_sf if pv_mode in ("bf16", "mxfp8") else None, meta_q, meta_k,
                  torch.bfloat16 if pv_mode == "bf16v" else torch.uint8)
    Tq, H = q.shape[0], q.shape[1]
    _check_out_lse(out, lse, meta_q.total_tokens, H, q.device)
    descs = []
    for name, t in (("q_descale", q_descale), ("k_descale", k_descale), ("v_descale", v_descale)):
        if t is None:
            descs.append(_Descale(None, 0, 0))
            continue
        ss, hs = descale_strides(t, meta_q.num_seqs, H)
        if debug_flags and (ss or hs):
            raise ValueError("the debug entry point takes per-tensor descales only")
        if t.device != q.device:
            raise ValueError("%s must be on the device of q" % name)
        descs.append(_Descale(t.data_ptr(), ss, hs))
    if out is None:
        out = torch.empty((Tq, H, 128), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((H, Tq), dtype=torch.float32, device=q.device)
    args = (q.data_ptr(), q_sf.data_ptr(), k.data_ptr(), k_sf.data_ptr(), v.data_ptr(), _ptr(v_sf),
            ctypes.byref(meta_q._c), ctypes.byref(meta_k._c), H, 128, PV_MODES[pv_mode],
            _ptr(q_descale), _ptr(k_descale), _ptr(v_descale), out.data_ptr(), lse.data_ptr(),
            _stream_ptr(stream))
    ws = None if debug_flags else _workspace(workspace, meta_k, H, pv_mode, q.device, stream)
    with torch.cuda.device(q.device):
        if debug_flags:
            _check(_lib.lpfa_attn_fwd_varlen_debug(*args, debug_flags))
        elif ws is not None:
            _check(_lib.lpfa_attn_fwd_varlen_ws(*args[:11], ctypes.byref(descs[0]), ctypes.byref(descs[1]),
                                                ctypes.byref(descs[2]), out.data_ptr(), lse.data_ptr(),
                                                ws.data_ptr(), ctypes.c_size_t(ws.numel()), _stream_ptr(stream)))
        else:
            _check(_lib.lpfa_attn_fwd_varlen_descaled(*args[:11], ctypes.byref(descs[0]), ctypes.byref(descs[1]),
                                                      ctypes.byref(descs[2]), *args[14:]))
    return out, lse


def lpfa_attn_fwd_workspace_bytes(meta_k: VarlenMeta, heads: int, pv_mode: str) -> int:
    """Workspace bytes the bf16 PV mode needs (Tk * H * 256); 0 for the other modes."""
    return int(_lib.lpfa_attn_fwd_workspace_bytes(ctypes.byref(meta_k._c), heads, PV_MODES[pv_mode]))


def _workspace(workspace, meta_k: VarlenMeta, heads: int, pv_mode: str, device, stream=None):
    """The workspace tensor for a forward call, or None (in-kernel V conversion / not needed)."""
    need = lpfa_attn_fwd_workspace_bytes(meta_k, heads, pv_mode)
    if need == 0 or workspace is False or workspace is None:
        return None
    if workspace is True:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        if isinstance(stream, torch.cuda.Stream):
            ws.record_stream(stream)  # the kernels read it on that stream after this call returns
        return ws
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be True, False or a contiguous uint8 device tensor")
    if workspace.numel() < need:
        raise ValueError("workspace has %d bytes; this call needs %d" % (workspace.numel(), need))
    return workspace


def lpfa_dequantize_mxfp8_varlen(payload: torch.Tensor, scales: torch.Tensor, meta: VarlenMeta,
                                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """MXFP8 (head_dim orientation) payload + scale storage -> BF16 (T, H, 128), exactly."""
    if payload.dtype != torch.uint8 or payload.dim() != 3 or not payload.is_contiguous():
        raise ValueError("payload must be a contiguous uint8 (tokens, heads, 128) tensor")
    T, H = payload.shape[0], payload.shape[1]
    if out is None:
        out = torch.empty((T, H, 128), dtype=torch.bfloat16, device=payload.device)
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (T, H, 128) or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 (tokens, heads, 128) tensor")
    with torch.cuda.device(payload.device):
        _check(_lib.lpfa_dequantize_mxfp8_varlen(payload.data_ptr(), scales.data_ptr(), ctypes.byref(meta._c), H,
                                                 128, out.data_ptr(), _stream_ptr(stream)))
    return out


def lpfa_attn_fwd_shared_q(q: torch.Tensor, q_sf: torch.Tensor, k: torch.Tensor, k_sf: torch.Tensor,
                           v: torch.Tensor, v_sf: Optional[torch.Tensor], meta_q: VarlenMeta, meta_k: VarlenMeta,
                           pv_mode: str = "bf16", q_descale: Optional[torch.Tensor] = None,
                           k_descale: Optional[torch.Tensor] = None, v_descale: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None,
                           workspace=True):
    """Shared-query forward (see include/lpfa.h): one query sequence (meta_q has one sequence of Lq
    tokens) attends to each of the n key/value sequences of meta_k. Returns (out bf16 (n*Lq,H,128),
    lse fp32 (H,n*Lq)); rows [i*Lq, (i+1)*Lq) belong to key/value sequence i. Descales and
    workspace as for lpfa_attn_fwd_varlen; descales are indexed by the key/value sequence."""
    if pv_mode not in PV_MODES:
        raise ValueError("pv_mode must be 'bf16', 'fp8', 'bf16v' or 'mxfp8'")
    if meta_q.num_seqs != 1:
        raise ValueError("a shared query set is one sequence")
    _check_packed(q, q_sf, k, k_sf, v, v_sf if pv_mode in ("bf16", "mxfp8") else None, meta_q, meta_k,
                  torch.bfloat16 if pv_mode == "bf16v" else torch.uint8)
    Lq, H = q.shape[0], q.shape[1]
    rows = Lq * meta_k.num_seqs
    descs = []
    for name, t in (("q_descale", q_descale), ("k_descale", k_descale), ("v_descale", v_descale)):
        if t is None:
            descs.append(_Descale(None, 0, 0))
            continue
        ss, hs = descale_strides(t, meta_k.num_seqs, H)
        if t.device != q.device:
            raise ValueError("%s must be on the device of q" % name)
        descs.append(_Descale(t.data_ptr(), ss, hs))
    if out is None:
        out = torch.empty((rows, H, 128), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((H, rows), dtype=torch.float32, device=q.device)
    if tuple(out.shape) != (rows, H, 128) or tuple(lse.shape) != (H, rows):
        raise ValueError("out must be (n*Lq, H, 128) and lse (H, n*Lq)")
    _check_out_lse(out, lse, rows, H, q.device)
    ws = _workspace(workspace, meta_k, H, pv_mode, q.device, stream)
    args = (q.data_ptr(), q_sf.data_ptr(), k.data_ptr(), k_sf.data_ptr(), v.data_ptr(), _ptr(v_sf),
            ctypes.byref(meta_q._c), ctypes.byref(meta_k._c), H, 128, PV_MODES[pv_mode], ctypes.byref(descs[0]),
            ctypes.byref(descs[1]), ctypes.byref(descs[2]), out.data_ptr(), lse.data_ptr())
    with torch.cuda.device(q.device):
        if ws is not None:
            _check(_lib.lpfa_attn_fwd_shared_q_ws(*args, ws.data_ptr(), ctypes.c_size_t(ws.numel()),
                                                  _stream_ptr(stream)))
        else:
            _check(_lib.lpfa_attn_fwd_shared_q(*args, _stream_ptr(stream)))
    return out, lse


def lpfa_attn_bwd_varlen(q: torch.Tensor, q_sf: torch.Tensor, k: torch.Tensor, k_sf: torch.Tensor,
                         v: torch.Tensor, v_sf: torch.Tensor, out: torch.Tensor, dout: torch.Tensor,
                         lse: torch.Tensor, meta_q: VarlenMeta, meta_k: VarlenMeta,
                         q_descale: Optional[torch.Tensor] = None, k_descale: Optional[torch.Tensor] = None,
                         v_descale: Optional[torch.Tensor] = None, output_mxfp8_dkv: bool = False, stream=None,
                         dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                         dv: Optional[torch.Tensor] = None, dk_sf: Optional[torch.Tensor] = None,
                         dv_sf: Optional[torch.Tensor] = None, debug_flags: int = 0):
    """Attention backward (see include/lpfa.h). q/k/v with their head_dim-orientation scales, out and
    dout bf16 (Tq,H,128), lse fp32 (H,Tq). Returns (dq, dk, dv) in bf16, or with output_mxfp8_dkv
    (dq, dk_payload, dv_payload, dk_scales, dv_scales) like LP-FA4's mxfp8_flash_attn_varlen_backward.
    Output tensors may be passed in (contiguous, of the returned shapes and dtypes); debug_flags != 0
    calls the test hook lpfa_attn_bwd_varlen_debug.
    """
    _check_packed(q, q_sf, k, k_sf, v, v_sf, meta_q, meta_k, torch.uint8)
    for name, t in (("out", out), ("dout", dout)):
        if t.dtype != torch.bfloat16 or t.shape != q.shape or not t.is_contiguous():
            raise ValueError("%s must be a contiguous bf16 tensor shaped like q" % name)
    Tq, H = q.shape[0], q.shape[1]
    Tk = k.shape[0]
    if lse.dtype != torch.float32 or tuple(lse.shape) != (H, Tq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (heads, tokens) tensor")
    descs = []
    for name, t in (("q_descale", q_descale), ("k_descale", k_descale), ("v_descale", v_descale)):
        if t is None:
            descs.append(_Descale(None, 0, 0))
        else:
            ss, hs = descale_strides(t, meta_q.num_seqs, H)
            descs.append(_Descale(t.data_ptr(), ss, hs))
    def _out(t, shape, dtype, name):
        if t is None:
            return torch.empty(shape, dtype=dtype, device=q.device)
        if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError("%s must be a contiguous %s tensor of shape %s" % (name, dtype, tuple(shape)))
        return t

    kv_dtype = torch.uint8 if output_mxfp8_dkv else torch.bfloat16
    dq = _out(dq, (Tq, H, 128), torch.bfloat16, "dq")
    dk = _out(dk, (Tk, H, 128), kv_dtype, "dk")
    dv = _out(dv, (Tk, H, 128), kv_dtype, "dv")
    if output_mxfp8_dkv:
        dk_sf = _out(dk_sf, (meta_k.scale_bytes(H),), torch.uint8, "dk_sf")
        dv_sf = _out(dv_sf, (meta_k.scale_bytes(H),), torch.uint8, "dv_sf")
    else:
        dk_sf = dv_sf = None
    args = (q.data_ptr(), q_sf.data_ptr(), k.data_ptr(), k_sf.data_ptr(), v.data_ptr(), v_sf.data_ptr(),
            out.data_ptr(), dout.data_ptr(), lse.data_ptr(), ctypes.byref(meta_q._c), ctypes.byref(meta_k._c), H, 128,
            ctypes.byref(descs[0]), ctypes.byref(descs[1]), ctypes.byref(descs[2]), dq.data_ptr(), dk.data_ptr(),
            dv.data_ptr(), _ptr(dk_sf), _ptr(dv_sf), 1 if output_mxfp8_dkv else 0, _stream_ptr(stream))
    with torch.cuda.device(q.device):
        if debug_flags:
            _check(_lib.lpfa_attn_bwd_varlen_debug(*args, int(debug_flags)))
        else:
            _check(_lib.lpfa_attn_bwd_varlen(*args))
    if output_mxfp8_dkv:
        return dq, dk, dv, dk_sf, dv_sf
    return dq, dk, dv


# ---------------------------------------------------------------------------------------
# Norm and rotation of Q and K
# ---------------------------------------------------------------------------------------
_DTYPE_CODE = {torch.bfloat16: 0, torch.float32: 1}
PAIRINGS = {"interleaved": 0, "half": 1}


class _Scope:
    """The device and stream of one call. Buffers made inside belong to the stream that the call's
    work runs on (its allocator pool), so neither earlier nor later work of another stream can share
    their memory; `seen_by_caller` marks results that the caller's own stream will go on to read."""

    __slots__ = ("device", "handle", "restore", "other", "caller")

    def __init__(self, device, stream):
        self.device = device
        self.restore = None if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)
        self.other = stream

    def __enter__(self):
        self.handle = torch._C._cuda_getCurrentRawStream(self.device.index)
        if self.other is not None:
            stream = self.other
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=self.device)
            elif stream.device != self.device:
                raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, self.device))
            self.other = None
            if stream.cuda_stream != self.handle:
                self.caller = torch.cuda.current_stream(self.device)
                self.handle, self.other = stream.cuda_stream, stream
        if self.restore is not None:  # last: what is refused above leaves the current device alone
            self.restore.__enter__()
        return self

    def __exit__(self, *exc):
        if self.restore is not None:
            self.restore.__exit__(*exc)

    def empty(self, shape, dtype, seen_by_caller=True):
        if self.other is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.other):
            t = torch.empty(shape, dtype=dtype, device=self.device)
        if seen_by_caller:
            t.record_stream(self.caller)
        return t

    def like(self, x, dtype):
        """A new contiguous tensor of x's shape."""
        if self.other is None:
            return torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)
        return self.empty(x.shape, dtype)


def _rows(t: torch.Tensor, name: str, dtype, index: int, shape=None) -> _Rows:
    """A (tokens, heads, 128) tensor on CUDA device `index` as an lpfa_rows."""
    s = t.shape
    if len(s) != 3 or s[2] != 128 or not s[0] or not s[1]:
        raise ValueError("%s must be a (tokens, heads, 128) tensor" % name)
    if t.dtype is not dtype or dtype not in _DTYPE_CODE:
        raise ValueError("%s must be %s" % (name, dtype if dtype in _DTYPE_CODE else "bf16 or fp32"))
    if index < 0 or t.get_device() != index:
        raise ValueError("%s must be on the CUDA device of the other tensors" % name)
    if shape is not None and s != shape:
        raise ValueError("%s must have shape %s" % (name, tuple(shape)))
    n, h, _ = s
    a, b, c = t.stride()
    if c != 1:
        raise ValueError("%s must have a contiguous last dimension" % name)
    # The stride of an axis of one element is never stepped over; it may be anything.
    return _Rows(t.data_ptr(), a if n > 1 else h * 128, b if h > 1 else 128, h)


def _out_rows(t: torch.Tensor, name: str, dtype, index, shape) -> _Rows:
    """As _rows, for a tensor that is written: its elements must be different memory."""
    r = _rows(t, name, dtype, index, shape)
    if t.is_contiguous():
        return r
    lo, hi = sorted(((r.tok_stride, shape[0]), (r.head_stride, shape[1])))
    if (lo[0] < 128 and lo[1] > 1) or (hi[1] > 1 and hi[0] < (lo[0] * (lo[1] - 1) + 128 if lo[1] > 1 else 128)):
        raise ValueError("%s has rows that overlap" % name)
    return r


def _contiguous(t: torch.Tensor, name: str, dtype, device, shape) -> torch.Tensor:
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != device:
        raise ValueError("%s must be a contiguous %s tensor of shape %s on the device of the others"
                         % (name, dtype, tuple(shape)))
    return t


class RotaryAxes:
    """How positions on one or more axes turn the 64 element pairs of a head.

    dims        head_dim elements given to each axis, even numbers with a sum of at most 128, e.g.
                (44, 42, 42) for time, height and width, or (128,) for text. Axis a owns the next
                dims[a] / 2 pairs, pair j of them with frequency theta[a] ** (-2 j / dims[a]). Pairs
                that no axis owns are left as they are.
    theta       one base for all axes, or one for each.
    pairing     "interleaved": pair i is elements (2i, 2i + 1); "half": (i, i + 64).

    from_frequencies takes any frequency and axis for each pair (scaled or shared spectra).
    """

    def __init__(self, dims: Sequence[int] = (128,), theta=10000.0, pairing: str = "interleaved"):
        dims = [int(d) for d in dims]
        thetas = [float(theta)] * len(dims) if np.ndim(theta) == 0 else [float(x) for x in theta]
        if not dims or any(d < 0 or d % 2 for d in dims) or sum(dims) > 128 or len(thetas) != len(dims):
            raise ValueError("dims must be even, sum to at most 128 and have one theta each (or one for all)")
        if any(not (x > 0) for x in thetas):
            raise ValueError("theta must be positive")
        freq, axis = [], []
        for a, (d, base) in enumerate(zip(dims, thetas)):
            for j in range(d // 2):
                freq.append(base ** (-2.0 * j / d))
                axis.append(a)
        freq += [0.0] * (64 - len(freq))
        axis += [0] * (64 - len(axis))
        self._fill(freq, axis, len(dims), pairing)

    @classmethod
    def from_frequencies(cls, inv_freq: Sequence[float], axis: Optional[Sequence[int]] = None,
                         pairing: str = "interleaved") -> "RotaryAxes":
        """inv_freq: radians per position step of each of the 64 pairs; axis: its position column (0)."""
        freq = [float(x) for x in inv_freq]
        ax = [0] * 64 if axis is None else [int(x) for x in axis]
        if len(freq) != 64 or len(ax) != 64 or min(ax) < 0:
            raise ValueError("a head has 64 pairs: give 64 frequencies and axes")
        self = cls.__new__(cls)
        self._fill(freq, ax, max(ax) + 1, pairing)
        return self

    def _fill(self, freq, axis, axes, pairing):
        if pairing not in PAIRINGS:
            raise ValueError("pairing must be 'interleaved' or 'half'")
        if not 1 <= axes <= 8:
            raise ValueError("a rotation has 1 to 8 axes")
        if not np.isfinite(freq).all():
            raise ValueError("frequencies must be finite")
        self.axes, self.pairing = axes, pairing
        self.inv_freq, self.axis = tuple(freq), tuple(axis)
        self._c = _Rotary(axes, PAIRINGS[pairing], (ctypes.c_double * 64)(*freq), (ctypes.c_uint8 * 64)(*axis))
        self._ptr = ctypes.pointer(self._c)


def _weight(w: torch.Tensor, name: str, heads: int, dtype, index: int):
    """(address, stride between heads) of a weight."""
    s = w.shape
    if s[-1] != 128 or (len(s) != 1 and s != (heads, 128)) or not w.is_contiguous() or w.get_device() != index:
        raise ValueError("%s must be a contiguous (128,) or (heads, 128) tensor on the device of q" % name)
    if w.dtype is not dtype or dtype not in _DTYPE_CODE:
        raise ValueError("weights must be bf16 or fp32, both the same")
    return w.data_ptr(), 128 if len(s) == 2 else 0


def _norm_rope_op(tokens, index, q_heads, k_heads, positions, rope, q_weight, k_weight, eps, norm) -> _NormRope:
    if norm and not (0.0 <= eps < float("inf")):
        raise ValueError("eps must be finite and >= 0")
    rotary, pos, pt, pa, p64 = None, None, 0, 0, 0
    if rope is not None:
        if not isinstance(rope, RotaryAxes):
            raise ValueError("rope must be a RotaryAxes or None")
        if positions is None:
            raise ValueError("a rotation needs positions")
        s = positions.shape
        two = len(s) == 2
        if not 1 <= len(s) <= 2 or s[0] != tokens or (s[1] if two else 1) < rope.axes:
            raise ValueError("positions must be (tokens, axes): %d tokens, %d axes" % (tokens, rope.axes))
        dt = positions.dtype
        if dt is torch.int64:
            p64 = 1
        elif dt is not torch.int32:
            raise ValueError("positions must be int32 or int64")
        if positions.get_device() != index:
            raise ValueError("positions must be on the device of q")
        rotary, pos = rope._ptr, positions.data_ptr()
        if two:
            pt, pa = positions.stride()
        else:
            pt = positions.stride(0)
    qw, qs, kw, ks, wdt = None, 0, None, 0, torch.bfloat16
    if q_weight is not None:
        wdt = q_weight.dtype
        qw, qs = _weight(q_weight, "q_weight", q_heads, wdt, index)
    if k_weight is not None:
        if not k_heads:
            raise ValueError("k_weight without k")
        if q_weight is None:
            wdt = k_weight.dtype
        kw, ks = _weight(k_weight, "k_weight", k_heads, wdt, index)
    return _NormRope(rotary, pos, pt, pa, p64, 1 if norm else 0, eps, qw, qs, kw, ks, _DTYPE_CODE[wdt])


def _qk_rows(q, k, index):
    """lpfa_rows of q and (None without it) k, and the number of k's heads."""
    dt = q.dtype
    qr = _rows(q, "q", dt, index)
    if k is None:
        return qr, None, 0
    kr = _rows(k, "k", dt, index)
    if k.shape[0] != q.shape[0]:
        raise ValueError("q and k must have the same tokens")
    return qr, kr, kr.heads


def lpfa_qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                      rope: Optional[RotaryAxes], q_weight: Optional[torch.Tensor] = None,
                      k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, norm: bool = True,
                      out_dtype: Optional[torch.dtype] = None, q_out: Optional[torch.Tensor] = None,
                      k_out: Optional[torch.Tensor] = None, stream=None):
    """Per-head RMS norm and rotary positions of Q and K in one launch; returns (q_out, k_out).

    q, k: (tokens, heads, 128) bf16 or fp32 with any strides (views of a joint projection included);
    their head counts may differ and k may be None. positions: (tokens, axes) int32 or int64, or
    (tokens,) for one axis. rope: a RotaryAxes, or None for no rotation. q_weight, k_weight: (128,) or
    (heads, 128), bf16 or fp32. norm=False leaves the norm out (the weight still applies).
    Outputs: out_dtype (the input's by default), contiguous unless given; an output may be its own input, of the same
    type and strides, and overlaps nothing else.
    """
    index = q.get_device()
    qr, kr, k_heads = _qk_rows(q, k, index)
    device, dt, shape = q.device, q.dtype, q.shape
    odt = dt if out_dtype is None else out_dtype
    if odt not in _DTYPE_CODE:
        raise ValueError("out_dtype must be bf16 or fp32")
    op = _norm_rope_op(shape[0], index, qr.heads, k_heads, positions, rope, q_weight, k_weight, eps, norm)
    ko = None
    with _Scope(device, stream) as sc:
        if q_out is None:
            q_out = sc.like(q, odt)
            qo = _Rows(q_out.data_ptr(), shape[1] * 128, 128, shape[1])
        else:
            qo = _out_rows(q_out, "q_out", odt, index, shape)
        if k is None:
            if k_out is not None:
                raise ValueError("k_out without k")
        elif k_out is None:
            k_out = sc.like(k, odt)
            ko = _Rows(k_out.data_ptr(), k_heads * 128, 128, k_heads)
        else:
            ko = _out_rows(k_out, "k_out", odt, index, k.shape)
        _check(_lib.lpfa_qk_norm_rope(qr, kr, _DTYPE_CODE[dt], shape[0], 128, op, qo, ko, _DTYPE_CODE[odt], sc.handle))
    return q_out, k_out


def lpfa_qk_norm_rope_mxfp8(q: torch.Tensor, k: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                            rope: Optional[RotaryAxes], meta: VarlenMeta, q_weight: Optional[torch.Tensor] = None,
                            k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, norm: bool = True,
                            scaling_mode: str = "rceil", q_payload: Optional[torch.Tensor] = None,
                            q_scales: Optional[torch.Tensor] = None, k_payload: Optional[torch.Tensor] = None,
                            k_scales: Optional[torch.Tensor] = None, stream=None):
    """lpfa_qk_norm_rope straight into the attention's input: returns (q_payload, q_scales, k_payload,
    k_scales) as lpfa_quantize_mxfp8_varlen lays them out (None for k without k). The bytes are those
    of lpfa_qk_norm_rope with fp32 outputs and the quantizer after it."""
    index = q.get_device()
    qr, kr, k_heads = _qk_rows(q, k, index)
    device, dt, T = q.device, q.dtype, q.shape[0]
    if T != meta.total_tokens:
        raise ValueError("q has %d tokens but the metadata describes %d" % (T, meta.total_tokens))
    if scaling_mode not in SCALING_MODES:
        raise ValueError("scaling_mode must be 'rceil' or 'floor'")
    if k is None and (k_payload is not None or k_scales is not None):
        raise ValueError("k_payload or k_scales without k")
    _check_meta_device(meta, device)
    op = _norm_rope_op(T, index, qr.heads, k_heads, positions, rope, q_weight, k_weight, eps, norm)
    with _Scope(device, stream) as sc:
        q_payload, q_scales = _mxfp8_out(sc, q, meta, q_payload, q_scales, "q")
        kp = ks = None
        if k is not None:
            k_payload, k_scales = _mxfp8_out(sc, k, meta, k_payload, k_scales, "k")
            kp, ks = k_payload.data_ptr(), k_scales.data_ptr()
        _check(_lib.lpfa_qk_norm_rope_mxfp8(qr, kr, _DTYPE_CODE[dt], 128, meta._c, op, SCALING_MODES[scaling_mode],
                                            q_payload.data_ptr(), q_scales.data_ptr(), kp, ks, sc.handle))
    return q_payload, q_scales, k_payload, k_scales


def _mxfp8_out(sc, x, meta, payload, scales, name):
    """Payload and scale storage for x, new or checked."""
    nb = meta.total_scale_blocks * x.shape[1] * 512
    if payload is None:
        payload = sc.like(x, torch.uint8)
    else:
        _contiguous(payload, name + "_payload", torch.uint8, x.device, x.shape)
    if scales is None:
        scales = sc.empty(nb, torch.uint8)
    else:
        _contiguous(scales, name + "_scales", torch.uint8, x.device, (nb,))
    return payload, scales


def lpfa_qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor], q: torch.Tensor,
                          k: Optional[torch.Tensor], positions: Optional[torch.Tensor], rope: Optional[RotaryAxes],
                          q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                          eps: float = 1e-6, norm: bool = True, dq: Optional[torch.Tensor] = None,
                          dk: Optional[torch.Tensor] = None, dq_weight: Optional[torch.Tensor] = None,
                          dk_weight: Optional[torch.Tensor] = None, stream=None):
    """Gradients of lpfa_qk_norm_rope: returns (dq, dk, dq_weight, dk_weight), None for what is absent.

    dq_out, dk_out: gradients of its outputs, in the inputs' dtype (the attention backward's dQ and dK
    for bf16); q, k and the rest as in the forward call. Weight gradients are fp32 in the weight's
    shape. dq may be dq_out's memory, dk dk_out's. Equal calls give equal bits.
    """
    index = q.get_device()
    qr, kr, k_heads = _qk_rows(q, k, index)
    device, dt, shape = q.device, q.dtype, q.shape
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out come together")
    gq = _rows(dq_out, "dq_out", dt, index, shape)
    gk = _rows(dk_out, "dk_out", dt, index, k.shape) if k is not None else None
    op = _norm_rope_op(shape[0], index, qr.heads, k_heads, positions, rope, q_weight, k_weight, eps, norm)
    with _Scope(device, stream) as sc:
        dq = sc.like(q, dt) if dq is None else dq
        dqr = _out_rows(dq, "dq", dt, index, shape)
        dkr = None
        if k is not None:
            dk = sc.like(k, dt) if dk is None else dk
            dkr = _out_rows(dk, "dk", dt, index, k.shape)
        elif dk is not None:
            raise ValueError("dk without k")
        dws = []
        for w, dw, name in ((q_weight, dq_weight, "dq_weight"), (k_weight, dk_weight, "dk_weight")):
            if w is None:
                if dw is not None:
                    raise ValueError("%s without its weight" % name)
                dws.append(None)
            else:
                dws.append(sc.like(w, torch.float32) if dw is None else
                           _contiguous(dw, name, torch.float32, device, w.shape))
        need = _lib.lpfa_qk_norm_rope_bwd_workspace_bytes(shape[1], k_heads, op)
        ws = sc.empty(need, torch.uint8, seen_by_caller=False) if need else None
        _check(_lib.lpfa_qk_norm_rope_bwd(gq, gk, qr, kr, _DTYPE_CODE[dt], shape[0], 128, op, dqr, dkr, _ptr(dws[0]),
                                          _ptr(dws[1]), _ptr(ws), need, sc.handle))
    return dq, dk, dws[0], dws[1]


# ---------------------------------------------------------------------------------------
# MXFP4 key/value cache
# ---------------------------------------------------------------------------------------
def _check_meta_device(meta: VarlenMeta, device) -> None:
    if meta.dev is None or meta.dev.device != device:
        raise ValueError("the metadata must have a device buffer on the device of the tensors")


class Kv4Cache:
    """Pages of K and V in MXFP4 (include/lpfa.h, lpfa_kv4_cache): k and v are (num_pages, heads,
    page_size, 64) uint8, k_scales and v_scales (num_pages, heads, page_size, 4) uint8. Which page
    belongs to whom is the caller's page table; a page is copied, shared or freed by index."""

    def __init__(self, num_pages: int, heads: int, page_size: int = 64, device="cuda"):
        if num_pages < 1 or heads < 1 or page_size not in (16, 32, 64, 128, 256):
            raise ValueError("a cache has pages and heads, and 16, 32, 64, 128 or 256 tokens per page")
        shape = (num_pages, heads, page_size)
        self._set(*[torch.zeros(shape + (n,), dtype=torch.uint8, device=device) for n in (64, 4, 64, 4)])

    @classmethod
    def from_tensors(cls, k: torch.Tensor, k_scales: torch.Tensor, v: torch.Tensor, v_scales: torch.Tensor) -> "Kv4Cache":
        """A cache over existing tensors of the shapes above (a server's own pool)."""
        self = cls.__new__(cls)
        self._set(k, k_scales, v, v_scales)
        return self

    # Not to be replaced: the calls use the addresses taken here.
    k = property(lambda self: self._tensors[0])
    k_scales = property(lambda self: self._tensors[1])
    v = property(lambda self: self._tensors[2])
    v_scales = property(lambda self: self._tensors[3])

    def _set(self, k, k_scales, v, v_scales):
        if k.dim() != 4 or k.shape[3] != 64 or k.shape[2] not in (16, 32, 64, 128, 256):
            raise ValueError("k must be (num_pages, heads, page_size, 64) with 16, 32, 64, 128 or 256 tokens per page")
        if k.device.type != "cuda":
            raise ValueError("the cache lives on a CUDA device")
        for name, t, n in (("k", k, 64), ("k_scales", k_scales, 4), ("v", v, 64), ("v_scales", v_scales, 4)):
            _contiguous(t, name, torch.uint8, k.device, tuple(k.shape[:3]) + (n,))
        self._tensors = (k, k_scales, v, v_scales)
        self.num_pages, self.heads, self.page_size = k.shape[0], k.shape[1], k.shape[2]
        self.device = k.device
        self._c = _Kv4Cache(k.data_ptr(), k_scales.data_ptr(), v.data_ptr(), v_scales.data_ptr(), *k.shape[:3])


def _page_table(t: torch.Tensor, num_seqs: int, index: int) -> _PageTable:
    s = t.shape
    if t.dtype is not torch.int32 or len(s) != 2 or s[0] != num_seqs or s[1] < 1:
        raise ValueError("page_table must be an int32 (sequences, pages) tensor: %d sequences" % num_seqs)
    a, b = t.stride()
    if b != 1 and s[1] > 1:
        raise ValueError("page_table must have contiguous rows")
    if t.get_device() != index:
        raise ValueError("page_table must be on the device of the cache")
    return _PageTable(t.data_ptr(), a, s[1])


def _seq_ints(t: Optional[torch.Tensor], name: str, num_seqs: int, index: int) -> Optional[int]:
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.shape != (num_seqs,) or not t.is_contiguous() or t.get_device() != index:
        raise ValueError("%s must be a contiguous int32 tensor of %d sequences on the device of the cache" % (name, num_seqs))
    return t.data_ptr()


def lpfa_kv4_write(k: torch.Tensor, v: torch.Tensor, cache: Kv4Cache, page_table: torch.Tensor, meta: VarlenMeta,
                   start: Optional[torch.Tensor] = None, scaling_mode: str = "rceil", stream=None) -> None:
    """Quantize the packed new tokens k, v (T, heads, 128) (bf16 or fp32) into the cache's pages.

    meta: the new tokens of each sequence; start: int32 tokens cached before (None: 0); page_table:
    int32 (sequences, pages), token p of sequence s is row p % page_size of page
    page_table[s, p // page_size]. A page index out of range, or a token beyond the table, is skipped
    and reported by lpfa_device_status. Two tokens of a call must not share a slot.
    """
    device = cache.device
    index = device.index
    kr = _rows(k, "k", k.dtype, index)
    vr = _rows(v, "v", k.dtype, index, k.shape)
    if k.shape[1] != cache.heads:
        raise ValueError("k has %d heads, the cache %d" % (k.shape[1], cache.heads))
    if k.shape[0] != meta.total_tokens:
        raise ValueError("k has %d tokens but the metadata describes %d" % (k.shape[0], meta.total_tokens))
    if scaling_mode not in SCALING_MODES:
        raise ValueError("scaling_mode must be 'rceil' or 'floor'")
    _check_meta_device(meta, device)
    num_seqs = meta.num_seqs
    table = _page_table(page_table, num_seqs, device.index)
    starts = _seq_ints(start, "start", num_seqs, device.index)
    with _Scope(device, stream) as sc:
        _check(_lib.lpfa_kv4_write(kr, vr, _DTYPE_CODE[k.dtype], 128, cache._c, table, starts, meta._c,
                                   SCALING_MODES[scaling_mode], sc.handle))


def lpfa_kv4_read(cache: Kv4Cache, page_table: torch.Tensor, meta: VarlenMeta, start: Optional[torch.Tensor] = None,
                  k_payload: Optional[torch.Tensor] = None, k_scales: Optional[torch.Tensor] = None,
                  v_payload: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None, stream=None):
    """The cached tokens start[i] .. start[i] + length_i (lengths from meta) as packed MXFP8 tensors,
    exactly: (k_payload, k_scales, v_payload, v_scales) in the quantizer's layout, for lpfa_attn_fwd_varlen
    (pv_mode "bf16"; without a mask, and Q with the cache's heads) or lpfa_dequantize_mxfp8_varlen."""
    device = cache.device
    _check_meta_device(meta, device)
    num_seqs = meta.num_seqs
    table = _page_table(page_table, num_seqs, device.index)
    starts = _seq_ints(start, "start", num_seqs, device.index)
    shape, nb = (meta.total_tokens, cache.heads, 128), (meta.total_scale_blocks * cache.heads * 512,)
    u8 = torch.uint8
    with _Scope(device, stream) as sc:
        k = sc.empty(shape, u8) if k_payload is None else _contiguous(k_payload, "k_payload", u8, device, shape)
        ks = sc.empty(nb, u8) if k_scales is None else _contiguous(k_scales, "k_scales", u8, device, nb)
        v = sc.like(k, u8) if v_payload is None else _contiguous(v_payload, "v_payload", u8, device, shape)
        vs = sc.like(ks, u8) if v_scales is None else _contiguous(v_scales, "v_scales", u8, device, nb)
        _check(_lib.lpfa_kv4_read(cache._c, table, starts, meta._c, 128, k.data_ptr(), ks.data_ptr(), v.data_ptr(),
                                  vs.data_ptr(), sc.handle))
    return k, ks, v, vs


def lpfa_attn_fwd_kv4(q: torch.Tensor, cache: Kv4Cache, page_table: torch.Tensor, kv_lens: torch.Tensor,
                      meta_q: VarlenMeta, causal: bool = False, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, stream=None):
    """Attention of a few query tokens per sequence over the MXFP4 cache; returns (out bf16
    (Tq, q_heads, 128), lse fp32 (q_heads, Tq)).

    q: bf16 (Tq, q_heads, 128), q_heads a multiple of the cache's heads, packed under meta_q. kv_lens:
    int32 per sequence, the cached tokens (this step's included; 0 gives O = 0, LSE = -inf). causal:
    query token j of L sees the first kv_lens - L + j + 1 keys, else all of them. The page table is as
    for lpfa_kv4_write. Any number of query tokens is right, but every 8 or 16 query rows (tokens times query
    heads of a key head) read the cache again. Chunks of a few hundred tokens with as many heads as the cache and no
    causal mask are faster through lpfa_kv4_read and lpfa_attn_fwd_varlen, which has neither grouped heads nor a mask.
    """
    device = cache.device
    index = device.index
    qr = _rows(q, "q", torch.bfloat16, index)
    Tq, H = q.shape[0], q.shape[1]
    if H % cache.heads:
        raise ValueError("%d query heads are not a multiple of the cache's %d" % (H, cache.heads))
    if Tq != meta_q.total_tokens:
        raise ValueError("q has %d tokens but the metadata describes %d" % (Tq, meta_q.total_tokens))
    _check_meta_device(meta_q, device)
    num_seqs = meta_q.num_seqs
    table = _page_table(page_table, num_seqs, index)
    if kv_lens is None:
        raise ValueError("kv_lens is needed")
    lens = _seq_ints(kv_lens, "kv_lens", num_seqs, index)
    with _Scope(device, stream) as sc:
        if out is None:
            out = sc.like(q, torch.bfloat16)
        else:
            _contiguous(out, "out", torch.bfloat16, device, q.shape)
        if lse is None:
            lse = sc.empty((H, Tq), torch.float32)
        else:
            _contiguous(lse, "lse", torch.float32, device, (H, Tq))
        _check(_lib.lpfa_attn_fwd_kv4(qr, 128, cache._c, table, lens, meta_q._c, 1 if causal else 0, out.data_ptr(),
                                      lse.data_ptr(), sc.handle))
    return out, lse


def lpfa_device_status(stream=None):
    """Synchronize `stream` and return (status, detail) of the device status word (then reset)."""
    detail = _i32(0)
    st = _lib.lpfa_device_status(_stream_ptr(stream), ctypes.byref(detail))
    return st, detail.value


# LP-FA4 README names.
Mxfp8VarlenMeta = VarlenMeta
quantize_mxfp8_varlen = lpfa_quantize_mxfp8_varlen
mxfp8_flash_attn_varlen_forward = lpfa_attn_fwd_varlen
mxfp8_flash_attn_varlen_backward = lpfa_attn_bwd_varlen
fa4_v_to_fp8 = lpfa_cast_e4m3
