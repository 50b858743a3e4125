"""Python binding of librfx (the C ABI in include/rfx.h).

Argument marshalling only: every step of the decode path runs in the HIP
kernels of librfx.so. PyTorch is used for device memory and streams; device
arguments are torch tensors (their data_ptr() is passed through) and the
stream defaults to torch's current stream.

The library must be built first (``python -m bit_block_quantized_amd.build``
or ``__graft_entry__.build()``); importing this package without it raises.
"""

from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

FP2, FP3, FP4 = 2, 3, 4
FORMATS = (FP2, FP3, FP4)
# Variant: fp16 scale and fp16 minimum per block (weight = s * c + m),
# GEMV entry points only.
FP2M = 12
# A tier above FP4: 32 int8 codes + an fp16 scale (34 B), GEMV entry points only.
Q8 = 8
# Variant: FP2 codes with two fp16 sub-scales, one per 16-weight half (12 B),
# GEMV entry points only.
FP2S = 16
# A 3-bit tier at about 3.3 bits per weight: FP3 codes + an e8m0 byte (13 B),
# GEMV entry points only.
FP3E = 13
VARIANT_FORMATS = (FP2M, Q8, FP2S, FP3E)

RFX_OK = 0
RFX_E_TIMEOUT = -7
_STATUS = {-1: "RFX_E_INVAL", -2: "RFX_E_ALIGN", -3: "RFX_E_RANGE", -4: "RFX_E_UNSUPPORTED",
           -5: "RFX_E_WORKSPACE", -6: "RFX_E_HIP", -7: "RFX_E_TIMEOUT"}

HERE = os.path.dirname(os.path.abspath(__file__))
LIBPATH = os.path.join(HERE, "librfx.so")


class RfxError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


class QMat(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("count", ctypes.c_int32), ("data", ctypes.c_void_p)]


class GemvJob(ctypes.Structure):
    _fields_ = [("W", QMat), ("q", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("xq", ctypes.c_void_p), ("xs", ctypes.c_void_p), ("xsum", ctypes.c_void_p),
                ("y", ctypes.c_void_p)]


MAX_GEMV_JOBS = 16


class MoeLayerC(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("gate", QMat), ("up", QMat), ("down", QMat),
                ("sh_gate", QMat), ("sh_up", QMat), ("sh_down", QMat),
                ("router_w", ctypes.c_void_p), ("router_b", ctypes.c_void_p),
                ("expert_data", ctypes.c_void_p)]


class KVCacheC(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class KVBatchC(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("n_tokens", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("table_stride", ctypes.c_int32), ("q_off", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p)]


class QkRopeC(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("inv_freq", ctypes.c_void_p), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("n_heads", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class KVPrefixC(ctypes.Structure):
    _fields_ = [("n_groups", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("max_len", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("seq_off", ctypes.c_void_p), ("len", ctypes.c_void_p)]


class NormC(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("delta", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("delta_stride", ctypes.c_int64), ("weight", ctypes.c_void_p), ("sum", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("xq", ctypes.c_void_p), ("xs", ctypes.c_void_p), ("xsum", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("q", ctypes.c_int32), ("cols", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class LoraMatC(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("resid", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("rows", ctypes.c_int32), ("reserved", ctypes.c_int32)]


LORA_MAX_MATS = 4


class LoraC(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("n_adapters", ctypes.c_int32), ("rank", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("n_tokens", ctypes.c_int32), ("n_mats", ctypes.c_int32), ("x", ctypes.c_void_p),
                ("x_stride", ctypes.c_int64), ("ids", ctypes.c_void_p), ("mats", LoraMatC * LORA_MAX_MATS)]


class LogprobC(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("q", ctypes.c_int32), ("n_vocab", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("logprob", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("entropy", ctypes.c_void_p),
                ("rank", ctypes.c_void_p), ("top_index", ctypes.c_void_p), ("top_logprob", ctypes.c_void_p)]


# Element types of queries, cache, attention output and logits.
F32, F16, BF16 = 0, 1, 2

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t

_SIGS = {
    "rfx_status_str": ([_I], ctypes.c_char_p),
    "rfx_last_error": ([], ctypes.c_char_p),
    "rfx_version": ([], ctypes.c_char_p),
    "rfx_block_bytes": ([_I], _I),
    "rfx_code_bytes": ([_I], _I),
    "rfx_scale_bytes": ([_I], _I),
    "rfx_quantize_block": ([_I, _P, _P], _I),
    "rfx_dequantize_block": ([_I, _P, _P], _I),
    "rfx_qmat_bytes": ([_I, _I64, _I64], _I64),
    "rfx_quantize_matrix": ([_I, _P, _I64, _I64, _P, _I], _I),
    "rfx_export_blocks": ([_I, _P, _I64, _I64, _P], _I),
    "rfx_import_blocks": ([_I, _P, _I64, _I64, _P], _I),
    "rfx_quantize_act": ([_P, _I, _I, _P, _P, _P, _P], _I),
    "rfx_gemv_workspace_bytes": ([_P, _I], _SZ),
    "rfx_gemv": ([_P, _P, _P, _P, _I, _P, _P, _SZ, _P], _I),
    "rfx_gemv_noalloc": ([_P, _P, _P, _P, _I, _P, _P], _I),
    "rfx_gemv_q1": ([_P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "rfx_gemv_q4": ([_P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "rfx_gemv_grouped_workspace_bytes": ([_P, _I], _SZ),
    "rfx_gemv_grouped": ([_P, _I, _P, _SZ, _P], _I),
    "rfx_debug_block_dots": ([_P, _P, _P, _I, _P, _P], _I),
    "rfx_read_reference": ([_P, _SZ, _P, _I, _P], _I),
    "rfx_moe_workspace_bytes": ([_P, _I, _I], _SZ),
    "rfx_moe_route_topk": ([_P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "rfx_moe_ffn": ([_P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "rfx_moe_forward": ([_P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, ctypes.c_uint, _P], _I),
    "rfx_moe_forward_single_launch": ([_P, _I, _I], _I),
    "rfx_moe_forward_status": ([_P, _I, _I, _P, _SZ, _P], _I),
    "rfx_moe_debug_hidden": ([_P, _I, _I, _P, _SZ, _P, _P, _P, _P], _I),
    "rfx_moe_debug_prefill": ([_P, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _I, _I, _P, _P, _P, _P, _P], _I),
    "rfx_gemm_workspace_bytes": ([_P, _I], _SZ),
    "rfx_gemm": ([_P, _P, _P, _P, _I, _P, _I, _P, _P, _P, _SZ, _P], _I),
    "rfx_qk_norm_rope": ([_P, _P, _P, _P, _P], _I),
    "rfx_attn_workspace_bytes": ([_P, _P, _I], _SZ),
    "rfx_attn": ([_P, _P, _P, _I, _F, _I, _I, _P, _I, _P, _SZ, _P], _I),
    "rfx_attn_shared_workspace_bytes": ([_P, _P, _P, _I], _SZ),
    "rfx_attn_shared": ([_P, _P, _P, _P, _I, _F, _P, _I, _P, _SZ, _P], _I),
    "rfx_add_rms_norm": ([_P, _P], _I),
    "rfx_lora_workspace_bytes": ([_I, _I, _I, _I, _I], _SZ),
    "rfx_lora_apply": ([_P, _P, _SZ, _P], _I),
    "rfx_token_logprobs_workspace_bytes": ([_I, _I, _I], _SZ),
    "rfx_token_logprobs": ([_P, _I64, _P, _P, _P, _SZ, _P], _I),
}

EXPORTED = tuple(_SIGS)

_lib = None


def lib():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBPATH):
        raise ImportError(f"{LIBPATH} is missing: build it with "
                          "`python -m bit_block_quantized_amd.build`")
    L = ctypes.CDLL(LIBPATH)
    for name, (args, res) in _SIGS.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def _check(st: int):
    if st != RFX_OK:
        raise RfxError(st, lib().rfx_last_error().decode())
    return st


def _check_nonneg(v: int):
    if v < 0:
        raise RfxError(v, lib().rfx_last_error().decode())
    return v


def _np_ptr(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p)


def _dptr(t):
    """Device pointer of a torch tensor (or an int address, or None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


class _Torch:
    """torch's types and calls that the binding uses on every call, looked up
    once (importing this package does not import torch)."""
    f32 = None

    @classmethod
    def load(cls):
        import torch
        cls.f64, cls.i32, cls.i8 = torch.float64, torch.int32, torch.int8
        cls.elem = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
        # the C function under torch.cuda.current_device, where torch has it (who has a GPU tensor has begun to use the GPU)
        cls.current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        cls.device_guard = torch.cuda.device
        # the handle itself, without a Stream object around it, where torch has that
        cls.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        cls.f32 = torch.float32

    @staticmethod
    def on_stream(stream):
        """torch's own work goes to this stream (of the current device) too:
        None, a Stream or a handle, as the entry points take them."""
        import torch
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream)
        return torch.cuda.stream(stream)


def _torch():
    if _Torch.f32 is None:
        _Torch.load()
    return _Torch


def _stream(stream):
    if stream is None:
        t = _torch()
        return t.raw_stream(t.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------------ host

def block_bytes(fmt):
    return lib().rfx_block_bytes(fmt)


def code_bytes(fmt):
    return lib().rfx_code_bytes(fmt)


def scale_bytes(fmt):
    return lib().rfx_scale_bytes(fmt)


def qmat_bytes(fmt, rows, cols) -> int:
    n = lib().rfx_qmat_bytes(fmt, rows, cols)
    if n < 0:
        _check(int(n))
    return int(n)


def quantize_block(fmt, w) -> np.ndarray:
    w = np.ascontiguousarray(w, np.float32)
    if w.shape != (32,):
        raise ValueError("a block is 32 weights")
    out = np.zeros(max(block_bytes(fmt), 1), np.uint8)
    _check(lib().rfx_quantize_block(fmt, _np_ptr(w), _np_ptr(out)))
    return out


def dequantize_block(fmt, blk) -> np.ndarray:
    blk = np.ascontiguousarray(blk, np.uint8)
    out = np.zeros(32, np.float32)
    _check(lib().rfx_dequantize_block(fmt, _np_ptr(blk), _np_ptr(out)))
    return out


def quantize_matrix(fmt, W, threads: int = 0, out: np.ndarray | None = None) -> np.ndarray:
    """fp32 [rows][cols] -> tiled device layout (host uint8 array)."""
    W = np.ascontiguousarray(W, np.float32)
    rows, cols = W.shape
    n = qmat_bytes(fmt, rows, cols)
    if out is None:
        out = np.empty(n, np.uint8)
    elif out.nbytes < n or not out.flags.c_contiguous:
        raise ValueError("output buffer too small or not contiguous")
    _check(lib().rfx_quantize_matrix(fmt, _np_ptr(W), rows, cols, _np_ptr(out), threads))
    return out


def export_blocks(fmt, tiled, rows, cols) -> np.ndarray:
    tiled = np.ascontiguousarray(tiled, np.uint8)
    out = np.zeros((rows, cols // 32, block_bytes(fmt)), np.uint8)
    _check(lib().rfx_export_blocks(fmt, _np_ptr(tiled), rows, cols, _np_ptr(out)))
    return out


def import_blocks(fmt, blocks) -> np.ndarray:
    blocks = np.ascontiguousarray(blocks, np.uint8)
    rows, nb, bb = blocks.shape
    out = np.empty(qmat_bytes(fmt, rows, nb * 32), np.uint8)
    _check(lib().rfx_import_blocks(fmt, _np_ptr(blocks), rows, nb * 32, _np_ptr(out)))
    return out


# ---------------------------------------------------------------- device

class DeviceQMat:
    """A tiled matrix (or a stack of `count` matrices) in device memory."""

    def __init__(self, fmt, rows, cols, data, count=1):
        self.fmt, self.rows, self.cols, self.count = fmt, rows, cols, count
        self.data = data  # torch uint8 tensor on the GPU (kept alive here)
        # the GPU it is on, None where it does not say (an address, an object with data_ptr() alone)
        self.index = data.get_device() if hasattr(data, "get_device") else None
        self.c = QMat(fmt, rows, cols, count, _dptr(data))
        self.c_ref = ctypes.byref(self.c)

    @classmethod
    def from_host(cls, fmt, rows, cols, tiled: np.ndarray, count=1, device="cuda"):
        import torch
        t = torch.from_numpy(np.ascontiguousarray(tiled)).to(device)
        return cls(fmt, rows, cols, t, count)

    def expert(self, e: int) -> "DeviceQMat":
        nb = qmat_bytes(self.fmt, self.rows, self.cols)
        return DeviceQMat(self.fmt, self.rows, self.cols, self.data[e * nb:(e + 1) * nb], 1)

    def ref(self):
        return ctypes.byref(self.c)


def quantize_act(x, xq, xs, xsum, stream=None):
    q, K = x.shape
    _check(lib().rfx_quantize_act(_dptr(x), q, K, _dptr(xq), _dptr(xs), _dptr(xsum),
                                  _stream(stream)))


def gemv_workspace_bytes(W: DeviceQMat, q: int) -> int:
    return int(lib().rfx_gemv_workspace_bytes(W.ref(), q))


def gemv(W: DeviceQMat, xq, xs, xsum, q, y, ws=None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().rfx_gemv(W.ref(), _dptr(xq), _dptr(xs), _dptr(xsum), q, _dptr(y), _dptr(ws),
                          ws_bytes, _stream(stream)))


def gemv_noalloc(W: DeviceQMat, xq, xs, xsum, q, y, stream=None):
    """rfx_gemv with the library's own per-GPU scratch (no workspace)."""
    _check(lib().rfx_gemv_noalloc(W.ref(), _dptr(xq), _dptr(xs), _dptr(xsum), q, _dptr(y), _stream(stream)))


def gemv_q1(W: DeviceQMat, xq, xs, xsum, y, ws=None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().rfx_gemv_q1(W.ref(), _dptr(xq), _dptr(xs), _dptr(xsum), _dptr(y), _dptr(ws),
                             ws_bytes, _stream(stream)))


def gemv_q4(W: DeviceQMat, xq, xs, xsum, y, ws=None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().rfx_gemv_q4(W.ref(), _dptr(xq), _dptr(xs), _dptr(xsum), _dptr(y), _dptr(ws),
                             ws_bytes, _stream(stream)))


ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3, 4
ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH}


def gemm_workspace_bytes(W: DeviceQMat, q: int) -> int:
    return int(lib().rfx_gemm_workspace_bytes(W.ref(), q))


def _room(t, name, dtype, nbytes, index):
    """Address of a contiguous tensor of this dtype and at least this size on
    the device of this index; an address or None as it is."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype is dtype and t.nbytes >= nbytes and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype or t.nbytes < nbytes:
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, {dtype} of {nbytes // t.element_size()} elements wanted")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    raise ValueError(f"{name}: on {t.device}, not GPU {index}")


def _workspace(ws, index):
    """Address and size of a workspace tensor on the device of this index."""
    if ws is None:
        return None, 0
    if ws.get_device() != index:
        raise ValueError(f"ws: on {ws.device}, not GPU {index}")
    if not ws.is_contiguous():
        raise ValueError("ws: not contiguous")
    return ws.data_ptr(), ws.nbytes


def gemm(W: DeviceQMat, xq, xs, xsum, q, y, bias=None, act=ACT_NONE, resid=None, ws=None, stream=None):
    """y = resid + act(W x + bias) for q columns (rfx_gemm), on W's device:
    its current stream unless one is given. xq int8 [q][cols], xs float32 and
    xsum int32 [q][cols / 32], bias float32 [rows], y and resid float32
    [q][rows], contiguous and at least as large; a bare address is taken as it
    is."""
    t = _torch()
    index = t.current_device() if W.index is None else W.index
    f32, codes, out = t.f32, q * W.cols, 4 * q * W.rows
    wp, wn = _workspace(ws, index)
    _call_on(index, stream, lib().rfx_gemm, W.c_ref, _room(xq, "xq", t.i8, codes, index), _room(xs, "xs", f32, codes // 8, index),
             _room(xsum, "xsum", t.i32, codes // 8, index), q, _room(bias, "bias", f32, 4 * W.rows, index), act,
             _room(resid, "resid", f32, out, index), _room(y, "y", f32, out, index), wp, wn)


def gemv_jobs(jobs):
    """[(W: DeviceQMat, q, xq, xs, xsum, y), ...] -> ctypes array of rfx_gemv_job."""
    arr = (GemvJob * len(jobs))()
    for i, (W, q, xq, xs, xsum, y) in enumerate(jobs):
        arr[i] = GemvJob(W.c, q, 0, _dptr(xq), _dptr(xs), _dptr(xsum), _dptr(y))
    return arr


def gemv_grouped_workspace_bytes(jobs) -> int:
    arr = jobs if isinstance(jobs, ctypes.Array) else gemv_jobs(jobs)
    return int(lib().rfx_gemv_grouped_workspace_bytes(arr, len(arr)))


def gemv_grouped(jobs, ws=None, stream=None):
    """Several independent GEMVs in one launch; jobs as for gemv_jobs (or
    its result, reusable across calls)."""
    arr = jobs if isinstance(jobs, ctypes.Array) else gemv_jobs(jobs)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().rfx_gemv_grouped(arr, len(arr), _dptr(ws), ws_bytes, _stream(stream)))


def debug_block_dots(W: DeviceQMat, xq, xsum, q, dots, stream=None):
    _check(lib().rfx_debug_block_dots(W.ref(), _dptr(xq), _dptr(xsum), q, _dptr(dots),
                                      _stream(stream)))


def read_reference(buf, out, stream=None):
    """Measurement aid: stream `buf` (a device tensor) once; out (int32 or
    uint32 device tensor) gets one XOR fold per workgroup."""
    _check(lib().rfx_read_reference(_dptr(buf), buf.numel() * buf.element_size(), _dptr(out), out.numel(),
                                    _stream(stream)))


# ------------------------------------------------------------------ MoE

def moe_workspace_bytes(layer, q: int, k: int) -> int:
    return int(lib().rfx_moe_workspace_bytes(layer.ref(), q, k))


def moe_route_topk(layer, x, q, k, topk_idx, topk_w, pairs_sorted, expert_off, xq, xs, xsum, ws,
                   stream=None):
    _check(lib().rfx_moe_route_topk(layer.ref(), _dptr(x), q, k, _dptr(topk_idx), _dptr(topk_w),
                                    _dptr(pairs_sorted), _dptr(expert_off), _dptr(xq), _dptr(xs),
                                    _dptr(xsum), _dptr(ws), ws.numel() * ws.element_size(),
                                    _stream(stream)))


def moe_ffn(layer, q, k, xq, xs, xsum, topk_idx, topk_w, pairs_sorted, expert_off, y, ws,
            resid=None, stream=None):
    _check(lib().rfx_moe_ffn(layer.ref(), q, k, _dptr(xq), _dptr(xs), _dptr(xsum), _dptr(topk_idx),
                             _dptr(topk_w), _dptr(pairs_sorted), _dptr(expert_off), _dptr(resid),
                             _dptr(y), _dptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


FORWARD_ONE_LAUNCH = 1


def moe_forward(layer, x, q, k, y, topk_idx, topk_w, pairs_sorted, expert_off, xq, xs, xsum, ws,
                resid=None, one_launch=False, stream=None):
    """moe_route_topk then moe_ffn in one call; one_launch: the single-launch
    layer kernel where moe_forward_single_launch says it can take the call."""
    _check(lib().rfx_moe_forward(layer.ref(), _dptr(x), q, k, _dptr(resid), _dptr(y), _dptr(topk_idx),
                                 _dptr(topk_w), _dptr(pairs_sorted), _dptr(expert_off), _dptr(xq), _dptr(xs),
                                 _dptr(xsum), _dptr(ws), ws.numel() * ws.element_size(),
                                 FORWARD_ONE_LAUNCH if one_launch else 0, _stream(stream)))


def moe_forward_single_launch(layer, q: int, k: int) -> bool:
    return bool(_check_nonneg(lib().rfx_moe_forward_single_launch(layer.ref(), q, k)))


def moe_forward_status(layer, q, k, ws, stream=None):
    """Raises RfxError(RFX_E_TIMEOUT) if a bounded wait of the one-launch
    layer kernel ran out since the last check (synchronizes the stream)."""
    _check(lib().rfx_moe_forward_status(layer.ref(), q, k, _dptr(ws), ws.numel() * ws.element_size(),
                                        _stream(stream)))


def moe_debug_hidden(layer, q, k, ws, h=None, hq=None, hs=None, stream=None):
    _check(lib().rfx_moe_debug_hidden(layer.ref(), q, k, _dptr(ws), ws.numel() * ws.element_size(), _dptr(h),
                                      _dptr(hq), _dptr(hs), _stream(stream)))


def moe_debug_prefill(layer, q, k, xq, xs, topk_w, pairs_sorted, expert_off, ws, probe_expert, probe_first,
                      h=None, dots_gate=None, dots_up=None, dots_down=None, stream=None):
    """Test hook of the prefill path: reruns gate/up and down with the fp32 h
    and one work item's block dots stored (see include/rfx.h)."""
    _check(lib().rfx_moe_debug_prefill(layer.ref(), q, k, _dptr(xq), _dptr(xs), _dptr(topk_w), _dptr(pairs_sorted),
                                       _dptr(expert_off), _dptr(ws), ws.numel() * ws.element_size(), probe_expert,
                                       probe_first, _dptr(h), _dptr(dots_gate), _dptr(dots_up), _dptr(dots_down),
                                       _stream(stream)))


# ------------------------------------------------------------ attention

def _elem(dtype):
    """RFX_F32 / RFX_F16 / RFX_BF16 of a torch dtype."""
    e = _torch().elem.get(dtype)
    if e is None:
        raise ValueError(f"element type {dtype}: float32, float16 or bfloat16")
    return e


def _int32(**values):
    """ctypes wraps what an int32 does not hold."""
    for name, v in values.items():
        if not -0x80000000 <= v <= 0x7fffffff:
            raise ValueError(f"{name} {v}: from -2^31, below 2^31")


def _want(t, name, dtype, shape, index):
    """Address of a contiguous tensor of this dtype and shape (a tuple) on
    the device of this index (-1: host memory)."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index:
        return t.data_ptr()
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, {dtype} {tuple(shape)} wanted")
    raise ValueError(f"{name}: not contiguous" if not t.is_contiguous() else f"{name}: on {t.device}, not GPU {index}")


def _call_on(index, stream, fn, *args):
    """fn(*args, stream) with the tensors' device current; the stream
    defaults to that device's current one."""
    if index < 0:
        raise ValueError("tensors in host memory: the kernels need GPU memory")
    t = _torch()
    if t.current_device() != index:
        with t.device_guard(index):
            return _check(fn(*args, _stream(stream)))
    return _check(fn(*args, t.raw_stream(index) if stream is None else _stream(stream)))


class DeviceKVCache:
    """The paged cache of one layer: k and v [n_pages][n_kv_heads][page_size]
    [head_dim], float16 or bfloat16 (kept alive here)."""

    def __init__(self, k, v):
        n_pages, n_kv_heads, page_size, head_dim = k.shape
        if _elem(k.dtype) == F32:
            raise ValueError("the cache is float16 or bfloat16")
        self.k, self.v = k, v
        self.dtype, self.device, self.index = k.dtype, k.device, k.get_device()
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = n_pages, n_kv_heads, page_size, head_dim
        self.c = KVCacheC(_elem(k.dtype), n_kv_heads, head_dim, page_size, n_pages, 0,
                          _want(k, "k", k.dtype, k.shape, self.index), _want(v, "v", k.dtype, k.shape, self.index))
        self.c_ref = ctypes.byref(self.c)

    @classmethod
    def empty(cls, n_pages, n_kv_heads, page_size, head_dim, dtype=None, device="cuda"):
        import torch
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        dtype = torch.bfloat16 if dtype is None else dtype
        return cls(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device))

    def ref(self):
        return ctypes.byref(self.c)


class KVBatch:
    """A batch of sequences with new tokens (rfx_kv_batch): int32 device
    tensors q_off [n_seq + 1], kv_len [n_seq] (new tokens included) and
    page_table [n_seq][pages]; n_tokens rows in the token arrays, at most
    max_q new tokens per sequence."""

    def __init__(self, q_off, kv_len, page_table, n_tokens, max_q):
        n_seq, stride = page_table.shape
        _int32(n_tokens=n_tokens, max_q=max_q)
        self.q_off, self.kv_len, self.page_table = q_off, kv_len, page_table
        self.n_seq, self.n_tokens, self.max_q = n_seq, n_tokens, max_q
        self.index = dev = page_table.get_device()
        i32 = _torch().i32
        self.c = KVBatchC(n_seq, n_tokens, max_q, stride, _want(q_off, "q_off", i32, (n_seq + 1,), dev),
                          _want(kv_len, "kv_len", i32, (n_seq,), dev),
                          _want(page_table, "page_table", i32, (n_seq, stride), dev))
        self.c_ref = ctypes.byref(self.c)

    def ref(self):
        return ctypes.byref(self.c)


def rope_inv_freq(rot_dim, base=10000.0):
    """Angles per position of the rot_dim / 2 rotated pairs, float64:
    base^(-2 i / rot_dim)."""
    return np.float64(base) ** (-np.arange(0, rot_dim, 2, dtype=np.float64) / rot_dim)


def _head_rows(t, name, shape, index):
    """Address and row stride of float32 [n_tokens][heads][dim]; rows may be
    part of longer ones (a fused projection's output)."""
    if t.dtype is not _Torch.f32 or t.shape != shape:
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, float32 {shape} wanted")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, not GPU {index}")
    if t.is_contiguous():
        return t.data_ptr(), shape[1] * shape[2]
    row, head, one = t.stride()
    if one != 1 or (head != shape[2] and shape[1] > 1):
        raise ValueError(f"{name}: heads of a row are not contiguous (strides {t.stride()})")
    return t.data_ptr(), row if shape[0] > 1 else shape[1] * shape[2]


def _want_vec(t, name, dtype, n, index):
    """Address of n contiguous elements, 0 for None."""
    if t is None:
        return 0
    if t.dtype is dtype and t.numel() == n and t.is_contiguous() and t.get_device() == index:
        return t.data_ptr()
    return _want(t, name, dtype, (n,), index)


# rfx_qk_rope, packed in one go: a ctypes structure's fields cost twice as much
_pack_qk_rope = struct.Struct("3P3q3Pf3i").pack


def qk_norm_rope(q, k, v, cache: DeviceKVCache, batch: KVBatch, q_out, inv_freq, q_weight=None, k_weight=None,
                 eps=1e-6, interleaved=False, stream=None):
    """Norm and rotation of the new tokens' queries (into q_out) and keys,
    keys and values appended to the cache. q, k, v: float32 [n_tokens][heads]
    [head_dim], rows may be strided; inv_freq: float64 device tensor
    [rot_dim / 2] (see rope_inv_freq); weights float32 [head_dim] or None."""
    T, D, Hk, dev = batch.n_tokens, cache.head_dim, cache.n_kv_heads, cache.index
    Hq = q.shape[1]
    kv_shape = (T, Hk, D)
    qp, qs = _head_rows(q, "q", (T, Hq, D), dev)
    kp, ks = _head_rows(k, "k", kv_shape, dev)
    vp, vs = _head_rows(v, "v", kv_shape, dev)
    if batch.index != dev:
        raise ValueError(f"batch on GPU {batch.index}, the cache is on GPU {dev}")
    half = inv_freq.numel()
    f32 = _Torch.f32
    args = _pack_qk_rope(qp, kp, vp, qs, ks, vs, _want_vec(inv_freq, "inv_freq", _Torch.f64, half, dev),
                         _want_vec(q_weight, "q_weight", f32, D, dev), _want_vec(k_weight, "k_weight", f32, D, dev),
                         eps, Hq, 2 * half, interleaved)
    _call_on(dev, stream, lib().rfx_qk_norm_rope, args, cache.c_ref, batch.c_ref,
             _want(q_out, "q_out", cache.dtype, (T, Hq, D), dev))


def attn_workspace_bytes(cache: DeviceKVCache, batch: KVBatch, n_heads: int) -> int:
    return int(lib().rfx_attn_workspace_bytes(cache.ref(), batch.ref(), n_heads))


def attn(q, cache: DeviceKVCache, batch: KVBatch, out, scale, window=0, sinks=0, ws=None, stream=None):
    """Attention of the batch's new tokens over the paged cache: q
    [n_tokens][n_heads][head_dim] in the cache's type, out the same shape in
    that type or float32; window > 0: only the last `window` keys and the
    first `sinks`."""
    dev = cache.index
    Hq = q.shape[1]
    shape = (batch.n_tokens, Hq, cache.head_dim)
    qp = _want(q, "q", cache.dtype, shape, dev)
    op = _want(out, "out", out.dtype, shape, dev)
    if batch.index != dev:
        raise ValueError(f"batch on GPU {batch.index}, the cache is on GPU {dev}")
    _int32(window=window, sinks=sinks)
    wp, wn = _workspace(ws, dev)
    _call_on(dev, stream, lib().rfx_attn, qp, cache.c_ref, batch.c_ref, Hq, scale, window, sinks, op, _elem(out.dtype),
             wp, wn)


class KVPrefix:
    """Groups of a batch's sequences that share a prefix (rfx_kv_prefix): int32
    device tensors seq_off [n_groups + 1] and length [n_groups]; max_tokens: the
    most new tokens of a group's sequences in all, max_len: the longest prefix."""

    def __init__(self, seq_off, length, max_tokens, max_len):
        _int32(max_tokens=max_tokens, max_len=max_len)
        n, i32 = length.numel(), _torch().i32
        self.seq_off, self.length, self.max_tokens, self.max_len = seq_off, length, max_tokens, max_len
        self.n_groups, self.index = n, length.get_device()
        self.c = KVPrefixC(n, max_tokens, max_len, 0, _want(seq_off, "seq_off", i32, (n + 1,), self.index),
                           _want(length, "length", i32, (n,), self.index))
        self.c_ref = ctypes.byref(self.c)

    def ref(self):
        return ctypes.byref(self.c)


def attn_shared_workspace_bytes(cache: DeviceKVCache, batch: KVBatch, prefix: KVPrefix, n_heads: int) -> int:
    return int(lib().rfx_attn_shared_workspace_bytes(cache.ref(), batch.ref(), prefix.ref(), n_heads))


def attn_shared(q, cache: DeviceKVCache, batch: KVBatch, prefix: KVPrefix, out, scale, ws=None, stream=None):
    """attn for a batch whose sequences share prefixes, without a window: a
    prefix is read once for its group (rfx_attn_shared)."""
    dev = cache.index
    Hq = q.shape[1]
    shape = (batch.n_tokens, Hq, cache.head_dim)
    qp = _want(q, "q", cache.dtype, shape, dev)
    op = _want(out, "out", out.dtype, shape, dev)
    if batch.index != dev or prefix.index != dev:
        raise ValueError(f"batch and prefix on GPU {batch.index} and {prefix.index}, the cache is on GPU {dev}")
    wp, wn = _workspace(ws, dev)
    _call_on(dev, stream, lib().rfx_attn_shared, qp, cache.c_ref, batch.c_ref, prefix.c_ref, Hq, scale, op, _elem(out.dtype),
             wp, wn)


# --------------------------------- norm, adapters, log probabilities

def _rows(t, name, shape, index):
    """Address and row stride of float32 [q][cols]; rows may be part of
    longer ones."""
    if t.dtype is not _Torch.f32 or t.shape != shape:
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, float32 {tuple(shape)} wanted")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, not GPU {index}")
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    row, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: elements of a row are not contiguous (strides {t.stride()})")
    return t.data_ptr(), row if shape[0] > 1 else shape[1]


# rfx_norm, packed in one go like rfx_qk_rope
_pack_norm = struct.Struct("2P2q6Pf3i").pack


def add_rms_norm(x, weight, eps, delta=None, out=None, y=None, xq=None, xs=None, xsum=None, stream=None):
    """h = x + delta into `out`, its RMS norm times weight (None: 1) into y,
    that row's 8-bit activations into xq, xs, xsum (rfx_add_rms_norm); what is
    None is not written. x, delta: float32 [q][cols], rows may be strided; out
    and y float32 [q][cols]; xq int8 [q][cols], xs float32 and xsum int32
    [q][cols / 32]."""
    t = _torch()
    f32, shape, dev = t.f32, x.shape, x.get_device()
    q, cols = shape
    # the checks of _rows and _want, which raise, for tensors that pass them, at half the cost
    if x.dtype is f32 and x.is_contiguous():
        xp, x_stride = x.data_ptr(), cols
    else:
        xp, x_stride = _rows(x, "x", shape, dev)
    dp = d_stride = wp = op = yp = qp = sp = np_ = 0
    if delta is not None:
        if delta.dtype is f32 and delta.shape == shape and delta.is_contiguous() and delta.get_device() == dev:
            dp, d_stride = delta.data_ptr(), cols
        else:
            dp, d_stride = _rows(delta, "delta", shape, dev)
    if weight is not None:
        if weight.dtype is f32 and weight.shape == (cols,) and weight.is_contiguous() and weight.get_device() == dev:
            wp = weight.data_ptr()
        else:
            wp = _want(weight, "weight", f32, (cols,), dev)
    if out is not None:
        if out.dtype is f32 and out.shape == shape and out.is_contiguous() and out.get_device() == dev:
            op = out.data_ptr()
        else:
            op = _want(out, "out", f32, shape, dev)
    if y is not None:
        if y.dtype is f32 and y.shape == shape and y.is_contiguous() and y.get_device() == dev:
            yp = y.data_ptr()
        else:
            yp = _want(y, "y", f32, shape, dev)
    if xq is not None:
        blocks = (q, cols // 32)
        if xq.dtype is t.i8 and xq.shape == shape and xq.is_contiguous() and xq.get_device() == dev:
            qp = xq.data_ptr()
        else:
            qp = _want(xq, "xq", t.i8, shape, dev)
        if xs is None or xsum is None:
            raise ValueError("xq without xs and xsum")
        sp = _want(xs, "xs", f32, blocks, dev)
        np_ = _want(xsum, "xsum", t.i32, blocks, dev)
    elif xs is not None or xsum is not None:
        raise ValueError("xs and xsum without xq")
    if q: # an empty tensor has no address
        args = _pack_norm(xp, dp, x_stride, d_stride, wp, op, yp, qp, sp, np_, eps, q, cols, 0)
        if dev >= 0 and stream is None and t.current_device() == dev:
            _check(lib().rfx_add_rms_norm(args, t.raw_stream(dev)))
        else:
            _call_on(dev, stream, lib().rfx_add_rms_norm, args)


class DeviceLora:
    """The low-rank adapters of one projection (kept alive here): a
    [n_adapters][rank][cols] and b [n_adapters][rows][rank] in float16 or
    bfloat16, scale float32 [n_adapters] (alpha / rank) or None for 1."""

    def __init__(self, a, b, scale=None):
        n, rank, cols = a.shape
        if a.dtype != b.dtype or _elem(a.dtype) == F32:
            raise ValueError(f"adapters in {a.dtype} and {b.dtype}: both float16 or both bfloat16")
        if not 8 <= rank <= 128 or rank % 8 or cols % 32 or not cols:
            raise ValueError(f"rank {rank} (a multiple of 8, at most 128), cols {cols} (a multiple of 32)")
        if b.dim() != 3:
            raise ValueError(f"b: {tuple(b.shape)}, {(n, 'rows', rank)} wanted")
        self.a, self.b, self.scale = a, b, scale
        self.n_adapters, self.rank, self.cols, self.rows = n, rank, cols, b.shape[1]
        self.index = a.get_device()
        self.pointers = (_want(a, "a", a.dtype, a.shape, self.index), _want(b, "b", a.dtype, (n, self.rows, rank), self.index),
                         0 if scale is None else _want(scale, "scale", _torch().f32, (n,), self.index))
        # what matrices of one call have in common
        self.kind = (_elem(a.dtype), n, rank, cols)


def lora_workspace_bytes(loras, n_tokens: int) -> int:
    """For calls of these adapters (of one rank and columns) over n_tokens."""
    first = loras[0]
    _int32(n_tokens=n_tokens)
    return int(lib().rfx_lora_workspace_bytes(n_tokens, first.rank, len(loras), first.cols, first.n_adapters))


# rfx_lora up to its matrices, and one of those
_pack_lora, _pack_lora_mat = struct.Struct("6iPqP").pack, struct.Struct("5P2i").pack
_LORA_BYTES = ctypes.sizeof(LoraC)


def lora(x, ids, loras, ys, resids=None, ws=None, stream=None):
    """y = resid + scale B (A x) with each token's adapter, for up to four
    matrices over the same x (rfx_lora_apply). x: float32 [n_tokens][cols],
    rows may be strided; ids int32 [n_tokens] on the device, a token whose id
    is outside 0..n_adapters - 1 having none; loras: DeviceLora of one type,
    rank, number and columns; ys float32 [n_tokens][rows]; resids the same
    shapes, an entry None for 0; resids None: ys are added to in place."""
    first = loras[0]
    dev, (T, _) = first.index, x.shape
    t = _torch()
    f32, kind = t.f32, first.kind
    n = len(loras)
    if n > LORA_MAX_MATS or len(ys) != n or (resids is not None and len(resids) != n):
        raise ValueError(f"{n} matrices (at most {LORA_MAX_MATS}), {len(ys)} results")
    xp, x_stride = _rows(x, "x", (T, first.cols), dev)
    args = [_pack_lora(*kind, T, n, xp, x_stride, _want(ids, "ids", t.i32, (T,), dev))]
    for m, y, r in zip(loras, ys, ys if resids is None else resids):
        if m is not first and (m.kind != kind or m.index != dev):
            raise ValueError(f"matrices of (type, adapters, rank, cols) {m.kind} on GPU {m.index} and {kind} on GPU {dev}")
        shape = (T, m.rows)
        yp = _want(y, "y", f32, shape, dev)
        args.append(_pack_lora_mat(*m.pointers, 0 if r is None else yp if r is y else _want(r, "resid", f32, shape, dev), yp, m.rows, 0))
    if T: # an empty tensor has no address
        wp, wn = _workspace(ws, dev)
        _call_on(dev, stream, lib().rfx_lora_apply, b"".join(args).ljust(_LORA_BYTES, b"\0"), wp, wn)


def token_logprobs_workspace_bytes(q: int, n_vocab: int, top_k: int) -> int:
    _int32(q=q, n_vocab=n_vocab, top_k=top_k)
    return int(lib().rfx_token_logprobs_workspace_bytes(q, n_vocab, top_k))


class LogprobBuffers:
    """What rfx_token_logprobs says of q rows of n_vocab logits: logprob and
    rank of the given tokens, lse and entropy [q], and the top_k largest
    logits' top_index and top_logprob [q][top_k]; with its workspace."""

    def __init__(self, q: int, n_vocab: int, top_k: int = 0, device="cuda"):
        import torch
        if q < 1 or n_vocab < 1 or not 0 <= top_k <= 64:
            raise ValueError(f"q {q}, n_vocab {n_vocab}, top_k {top_k}")
        need = token_logprobs_workspace_bytes(q, n_vocab, top_k)
        if not need:
            raise ValueError(f"q {q} (at most 65536), n_vocab {n_vocab} (at most 2^19)")

        def empty(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=device)

        self.q, self.n_vocab, self.top_k = q, n_vocab, top_k
        self.logprob, self.lse, self.entropy = empty(q), empty(q), empty(q)
        self.rank = empty(q, dtype=torch.int32)
        self.top_index, self.top_logprob = empty(q, top_k, dtype=torch.int32), empty(q, top_k)
        self.ws = empty(need, dtype=torch.uint8)
        self.index = self.ws.get_device()
        top = [t.data_ptr() if top_k else None for t in (self.top_index, self.top_logprob)]
        rest = [t.data_ptr() for t in (self.logprob, self.lse, self.entropy, self.rank)]
        # per type, with tokens and without
        self._c = {d: (LogprobC(e, q, n_vocab, top_k, *rest, *top), LogprobC(e, q, n_vocab, top_k, None, *rest[1:3], None, *top))
                   for d, e in _torch().elem.items()}

    def run(self, logits, tokens=None, stream=None):
        """logits [q][n_vocab] in float32, float16 or bfloat16, rows may be
        strided; tokens int32 [q], a token outside 0..n_vocab - 1 being none,
        or None: then logprob and rank keep what they hold."""
        c, dev = self._c.get(logits.dtype), self.index
        if c is None or logits.shape != (self.q, self.n_vocab):
            raise ValueError(f"logits: {logits.dtype} {tuple(logits.shape)}, {(self.q, self.n_vocab)} in float32, float16 or "
                             "bfloat16 wanted")
        if logits.get_device() != dev:
            raise ValueError(f"logits: on {logits.device}, not GPU {dev}")
        row, one = logits.stride()
        if one != 1 and self.n_vocab > 1:
            raise ValueError(f"logits: elements of a row are not contiguous (strides {logits.stride()})")
        if tokens is not None:
            tokens = _want(tokens, "tokens", _torch().i32, (self.q,), dev)
        _call_on(dev, stream, lib().rfx_token_logprobs, logits.data_ptr(), row if self.q > 1 else self.n_vocab, tokens,
                 ctypes.byref(c[tokens is None]), self.ws.data_ptr(), self.ws.nbytes)
        return self


from .layer import (AttentionBuffers, DeviceAttention, DeviceHead, DeviceMoeLayer, HeadBuffers, MoeBuffers,  # noqa: E402,F401
                    PlacedMoeLayer, hot_experts_by_frequency)
from . import layer  # noqa: E402,F401
