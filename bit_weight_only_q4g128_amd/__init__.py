"""Python binding of libq4gemv.so (4-bit weight-only dequant-GEMV for gfx950).

Argument marshalling only: every step runs in the HIP library.  Tensors must
be CUDA (ROCm) tensors, contiguous (tokens of heads may lie apart, where a
function says so), with the dtypes the C header documents;
calls are enqueued on torch's current stream of the tensors' device.  There is
no CPU fallback: importing fails loudly if the library has not been built
(``python bit_weight_only_q4g128_amd/_build.py``).
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

__all__ = [
    "q4g128_gemv", "q4g128_gemv_grouped", "q4g128_gemv_grouped_noalloc", "NOALLOC_SCRATCH_BYTES", "nvfp4g16_gemv", "bf16_gemv", "q4g128_dequant_f32", "nvfp4g16_dequant_f32",
    "nvfp4g16_gemv_grouped", "nvfp4g16_workspace_bytes", "bf16_gemv_grouped", "bf16_workspace_bytes",
    "q4g128_gemv_fused", "q4g128_fused_workspace_bytes", "sample_topk", "bf16_head_sample", "bf16_head_sample_workspace_bytes", "q4g128_gemm", "gemv_grouped_mixed", "mixed_workspace_bytes",
    "fp8b128_quantize", "fp8b128_gemm", "fp8b128_gemm_grouped", "fp8b128_workspace_bytes",
    "verify_topk", "verify_topk_workspace_bytes", "verify_full", "verify_full_workspace_bytes",
    "rope_cache", "attention_decode", "attention_decode_workspace_bytes", "attention_prefill",
    "variant_name", "strerror", "Q4GemvError", "LIB_PATH", "lib", "stream_read", "stream_read_sink_words",
    "VARIANT_AUTO", "VARIANT_DOT2", "VARIANT_MFMA", "VARIANT_STREAM", "VARIANT_TILED", "VARIANT_GEMM", "FMT_Q4G128", "FMT_NVFP4G16", "FMT_BF16",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libq4gemv.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing; build it with: python bit_weight_only_q4g128_amd/_build.py")
lib = ctypes.CDLL(LIB_PATH)

VARIANT_AUTO, VARIANT_DOT2, VARIANT_MFMA, VARIANT_STREAM, VARIANT_TILED, VARIANT_GEMM = 0, 1, 2, 3, 4, 5
FMT_Q4G128, FMT_NVFP4G16, FMT_BF16 = 0, 1, 2

_p, _i, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
lib.q4g128_gemv_variant.argtypes = [_p, _i, _i, _p, _p, _p, _i, _p, _i, _p]
lib.q4g128_gemm_variant.argtypes = [_p, _i, _i, _p, _p, _p, _i, _p, _i, _p]
lib.nvfp4g16_gemv_variant.argtypes = [_p, _i, _i, _p, _p, _f, _i, _p, _i, _p]
lib.bf16_gemv_variant.argtypes = [_p, _i, _i, _p, _i, _p, _i, _p]
lib.q4g128_gemv.argtypes = [_p, _i, _i, _p, _p, _p, _i, _p, _p]
lib.nvfp4g16_gemv.argtypes = [_p, _i, _i, _p, _p, _f, _i, _p, _p]
lib.bf16_gemv.argtypes = [_p, _i, _i, _p, _i, _p, _p]
lib.q4g128_dequant_f32.argtypes = [_p, _p, _p, _i, _i, _p, _p]
lib.nvfp4g16_dequant_f32.argtypes = [_p, _p, _f, _i, _i, _p, _p]
for _fn in ("q4g128_gemv_variant", "nvfp4g16_gemv_variant", "bf16_gemv_variant", "q4g128_gemv", "nvfp4g16_gemv",
            "bf16_gemv", "q4g128_dequant_f32", "nvfp4g16_dequant_f32"):
    getattr(lib, _fn).restype = ctypes.c_int
lib.q4gemv_variant_name.argtypes = [_i, _i, _i, _i, _i]
lib.q4gemv_variant_name.restype = ctypes.c_char_p
lib.q4gemv_strerror.argtypes = [_i]
lib.q4gemv_strerror.restype = ctypes.c_char_p
lib.q4gemv_time_next_launch.argtypes = [_p, _p]
lib.q4gemv_time_next_launch.restype = ctypes.c_int
lib.q4gemv_version.argtypes = []
lib.q4gemv_version.restype = ctypes.c_int
lib.q4gemv_stream_read.argtypes = [ctypes.POINTER(_p), ctypes.POINTER(ctypes.c_size_t), _i, _p, ctypes.c_size_t, _p]
lib.q4gemv_stream_read.restype = ctypes.c_int
lib.q4gemv_stream_read_sink_words.argtypes = [ctypes.POINTER(ctypes.c_size_t), _i]
lib.q4gemv_stream_read_sink_words.restype = ctypes.c_size_t


class Q4Task(ctypes.Structure):
    """Mirror of the C struct q4g128_task."""
    _fields_ = [("x", _p), ("qweight", _p), ("scale", _p), ("minv", _p), ("y", _p), ("N", _i), ("K", _i)]


lib.q4g128_gemv_grouped.argtypes = [ctypes.POINTER(Q4Task), _i, _i, _i, _p]
lib.q4g128_gemv_grouped.restype = ctypes.c_int
lib.q4g128_gemv_grouped_ws.argtypes = [ctypes.POINTER(Q4Task), _i, _i, _i, _p, ctypes.c_size_t, _p]
lib.q4g128_gemv_grouped_ws.restype = ctypes.c_int
lib.q4g128_workspace_bytes.argtypes = [ctypes.POINTER(Q4Task), _i, _i, ctypes.POINTER(ctypes.c_size_t)]
lib.q4g128_gemv_grouped_noalloc.argtypes = [ctypes.POINTER(Q4Task), _i, _i, _i, _p]
lib.q4g128_gemv_grouped_noalloc.restype = ctypes.c_int
NOALLOC_SCRATCH_BYTES = 8 << 20
lib.q4g128_workspace_bytes.restype = ctypes.c_int


class NvTask(ctypes.Structure):
    """Mirror of the C struct nvfp4g16_task."""
    _fields_ = [("x", _p), ("qweight", _p), ("scale_e4m3", _p), ("global_scale", _f), ("y", _p), ("N", _i), ("K", _i)]


class BfTask(ctypes.Structure):
    """Mirror of the C struct bf16_task."""
    _fields_ = [("x", _p), ("w", _p), ("y", _p), ("N", _i), ("K", _i)]


for _name, _T in (("nvfp4g16", NvTask), ("bf16", BfTask)):
    getattr(lib, f"{_name}_gemv_grouped_ws").argtypes = [ctypes.POINTER(_T), _i, _i, _i, _p, ctypes.c_size_t, _p]
    getattr(lib, f"{_name}_gemv_grouped_ws").restype = ctypes.c_int
    getattr(lib, f"{_name}_workspace_bytes").argtypes = [ctypes.POINTER(_T), _i, _i, ctypes.POINTER(ctypes.c_size_t)]
    getattr(lib, f"{_name}_workspace_bytes").restype = ctypes.c_int


class FusedTask(ctypes.Structure):
    _fields_ = [("x", _p), ("up", _p), ("qweight", _p), ("scale", _p), ("minv", _p), ("residual", _p), ("y", _p),
                ("N", _i), ("K", _i)]


lib.q4g128_gemv_fused.argtypes = [ctypes.POINTER(FusedTask), _i, _i, _p, ctypes.c_size_t, _p]
lib.q4g128_gemv_fused.restype = ctypes.c_int
lib.q4g128_fused_workspace_bytes.argtypes = [ctypes.POINTER(FusedTask), _i, _i, ctypes.POINTER(ctypes.c_size_t)]
lib.q4g128_fused_workspace_bytes.restype = ctypes.c_int


class MixedTask(ctypes.Structure):
    _fields_ = [("format", _i), ("x", _p), ("weight", _p), ("scale", _p), ("minv", _p), ("global_scale", _f), ("y", _p),
                ("N", _i), ("K", _i)]


lib.q4gemv_grouped_mixed.argtypes = [ctypes.POINTER(MixedTask), _i, _i, _p, ctypes.c_size_t, _p]
lib.q4gemv_grouped_mixed.restype = ctypes.c_int
lib.q4gemv_mixed_workspace_bytes.argtypes = [ctypes.POINTER(MixedTask), _i, _i, ctypes.POINTER(ctypes.c_size_t)]
lib.q4gemv_mixed_workspace_bytes.restype = ctypes.c_int
lib.q4g128_gemm.argtypes = [_p, _i, _i, _p, _p, _p, _i, _p, _p]
lib.q4g128_gemm.restype = ctypes.c_int
lib.q4_sample_topk.argtypes = [_p, _i, _i, _f, _i, _p, _p, _p, _p, _p]
lib.q4_sample_topk.restype = ctypes.c_int
lib.bf16_head_sample.argtypes = [_p, _i, _i, _p, _i, _p, _f, _i, _p, _p, _p, _p, _p]
lib.bf16_head_sample.restype = ctypes.c_int
lib.bf16_head_sample_ws.argtypes = [_p, _i, _i, _p, _i, _p, _f, _i, _p, _p, _p, _p, _p, ctypes.c_size_t, _p]
lib.bf16_head_sample_ws.restype = ctypes.c_int
lib.bf16_head_sample_workspace_bytes.argtypes = [_i, _i, _i, _i]
lib.bf16_head_sample_workspace_bytes.restype = ctypes.c_size_t




class Fp8Task(ctypes.Structure):
    """Mirror of the C struct fp8b128_task (an array of them, or its bytes)."""
    _fields_ = [("x", _p), ("xscale", _p), ("w", _p), ("wscale", _p), ("residual", _p), ("y", _p), ("N", _i), ("K", _i)]


class Fp8Launch(ctypes.Structure):
    """Mirror of the C struct fp8b128_launch."""
    _fields_ = [("tile_m", _i), ("tile_n", _i), ("count", _i), ("N", _i * 8), ("slices", _i * 8), ("workspace_bytes", ctypes.c_size_t)]


lib.fp8b128_quantize.argtypes = [_p, _p, _i, _i, _p, _p, _p]
lib.fp8b128_quantize.restype = ctypes.c_int
lib.fp8b128_gemm.argtypes = [_p, _p, _i, _i, _p, _p, _i, _p, _p, _p]
lib.fp8b128_gemm.restype = ctypes.c_int
lib.fp8b128_gemm_grouped_ws.argtypes = [_p, _i, _i, _p, ctypes.c_size_t, _p]
lib.fp8b128_gemm_grouped_ws.restype = ctypes.c_int
lib.fp8b128_workspace_bytes.argtypes = [_p, _i, _i, ctypes.POINTER(ctypes.c_size_t)]
lib.fp8b128_workspace_bytes.restype = ctypes.c_int
lib.fp8b128_launches.argtypes = [_p, _i, _i, ctypes.c_size_t, _p, _i, ctypes.POINTER(_i)]
lib.fp8b128_launches.restype = ctypes.c_int
lib.q4_verify_topk.argtypes = [_p, _i, _i, _i, _p, _p, _p, _i, _p, _p, _f, _i, _p, _p, _p, _p, ctypes.c_size_t, _p]
lib.q4_verify_topk.restype = ctypes.c_int
lib.q4_verify_topk_workspace_bytes.argtypes = [_i, _i, _i, _i]
lib.q4_verify_topk_workspace_bytes.restype = ctypes.c_size_t
lib.q4_verify_full.argtypes = [_p, _i, _i, _i, _p, _p, _p, _p, _f, _p, _p, _p, _p, ctypes.c_size_t, _p]
lib.q4_verify_full.restype = ctypes.c_int
lib.q4_verify_full_workspace_bytes.argtypes = [_i, _i, _i]
lib.q4_verify_full_workspace_bytes.restype = ctypes.c_size_t
_l = ctypes.c_int64
lib.q4_rope_cache.argtypes = [_p, _p, _p, _i, _i, _i, _i, _l, _l, _l, _p, _p, _f, _p, _p, _i, _i, _p, _p, _p, _p, _p]
lib.q4_rope_cache.restype = ctypes.c_int
lib.q4_attention_decode_workspace_bytes.argtypes = [_i, _i, _i, _i]
lib.q4_attention_decode_workspace_bytes.restype = ctypes.c_size_t
lib.q4_attention_decode.argtypes = [_p, _i, _i, _i, _i, _i, _l, _p, _p, _i, _p, _p, _f, _i, _p, _p, ctypes.c_size_t, _p]
lib.q4_attention_decode.restype = ctypes.c_int
lib.q4_attention_prefill.argtypes = [_p, _i, _p, _p, _i, _i, _i, _i, _l, _l, _l, _p, _p, _i, _f, _i, _p, _p]
lib.q4_attention_prefill.restype = ctypes.c_int


class Q4GemvError(ValueError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(f"q4gemv status {status}: {strerror(status)}")


def strerror(status: int) -> str:
    return lib.q4gemv_strerror(int(status)).decode()


def variant_name(fmt: int, variant: int, M: int, N: int, K: int) -> str:
    return lib.q4gemv_variant_name(fmt, variant, M, N, K).decode()


def _check(t: torch.Tensor, name: str, dtypes, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _out(out, shape, dtype, like):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _check(out, "out", (dtype,), len(shape))
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(shape)}")
    return out


def _raise(rc: int):
    if rc != 0:
        raise Q4GemvError(rc)


_U16 = (torch.bfloat16, torch.int16)
_F16 = (torch.float16, torch.int16)
_U8 = (torch.uint8,)
_E4M3 = (torch.uint8, torch.float8_e4m3fn)


def q4g128_gemv(x, qweight, scale, minv, out=None, variant: int = VARIANT_AUTO):
    """y[M, N] = x[M, K] . W^T, W int4 g128 min/max (qweight uint8 [N, K/2],
    scale/min fp16 [N, K/128])."""
    _check(x, "x", _U16, 2); _check(qweight, "qweight", _U8, 2)
    _check(scale, "scale", _F16, 2); _check(minv, "min", _F16, 2)
    M, K = x.shape
    N = qweight.shape[0]
    if qweight.shape[1] * 2 != K or tuple(scale.shape) != (N, K // 128) or tuple(minv.shape) != (N, K // 128):
        raise ValueError("inconsistent shapes")
    y = _out(out, (M, N), torch.bfloat16, x)
    _raise(lib.q4g128_gemv_variant(x.data_ptr(), M, K, qweight.data_ptr(), scale.data_ptr(), minv.data_ptr(), N,
                                   y.data_ptr(), int(variant), _stream(x)))
    return y


def _task_array(items):
    items = list(items)
    if not 1 <= len(items) <= 8:
        raise ValueError("1..8 tasks per call")
    arr = (Q4Task * len(items))()
    outs = []
    M = None
    for i, (x, qweight, scale, minv, out) in enumerate(items):
        _check(x, "x", _U16, 2); _check(qweight, "qweight", _U8, 2)
        _check(scale, "scale", _F16, 2); _check(minv, "min", _F16, 2)
        m, K = x.shape
        N = qweight.shape[0]
        if M is None:
            M = m
        if m != M:
            raise ValueError("all tasks must share the batch size M")
        if qweight.shape[1] * 2 != K or tuple(scale.shape) != (N, K // 128) or tuple(minv.shape) != (N, K // 128):
            raise ValueError(f"task {i}: inconsistent shapes")
        y = _out(out, (M, N), torch.bfloat16, x)
        outs.append(y)
        arr[i] = Q4Task(x.data_ptr(), qweight.data_ptr(), scale.data_ptr(), minv.data_ptr(), y.data_ptr(), N, K)
    return items, arr, outs, M


def q4g128_gemv_grouped(items, variant: int = VARIANT_AUTO, workspace=None):
    """Several independent int4 g128 GEMVs with one batch size, launched
    together.  items: sequence of (x, qweight, scale, min, out-or-None).
    workspace: optional uint8 device tensor of at least
    q4g128_workspace_bytes(items) bytes, zero-filled before its first use and
    reusable afterwards without clearing (lets large batches split K).
    Returns the list of outputs."""
    items, arr, outs, M = _task_array(items)
    st = _stream(items[0][0])
    if workspace is None:
        _raise(lib.q4g128_gemv_grouped(arr, len(items), M, int(variant), st))
    else:
        if workspace.device != items[0][0].device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the activations' device")
        _raise(lib.q4g128_gemv_grouped_ws(arr, len(items), M, int(variant), workspace.data_ptr(), workspace.numel(), st))
    return outs


def q4g128_gemv_grouped_noalloc(items, variant: int = VARIANT_AUTO):
    """q4g128_gemv_grouped with the library's built-in split-K scratch instead
    of a workspace (q4g128_gemv_grouped_noalloc in the C header: nothing is
    allocated; calls on one GPU must not overlap in time).  items as for
    q4g128_gemv_grouped.  Returns the list of outputs."""
    items, arr, outs, M = _task_array(items)
    _raise(lib.q4g128_gemv_grouped_noalloc(arr, len(items), M, int(variant), _stream(items[0][0])))
    return outs


def q4g128_workspace_bytes(items) -> int:
    """Bytes of zero-filled workspace q4g128_gemv_grouped may use for these
    tasks (0: it never splits them)."""
    items, arr, _, M = _task_array(items)
    n = ctypes.c_size_t(0)
    _raise(lib.q4g128_workspace_bytes(arr, len(items), M, ctypes.byref(n)))
    return int(n.value)


def nvfp4g16_gemv(x, qweight, scale_e4m3, global_scale: float, out=None, variant: int = VARIANT_AUTO):
    """y[M, N] = x . W^T, W NVFP4 (qweight uint8 [N, K/2] E2M1, scale_e4m3
    [N, K/16], global_scale fp32 multiplier)."""
    _check(x, "x", _U16, 2); _check(qweight, "qweight", _U8, 2); _check(scale_e4m3, "scale_e4m3", _E4M3, 2)
    M, K = x.shape
    N = qweight.shape[0]
    if qweight.shape[1] * 2 != K or tuple(scale_e4m3.shape) != (N, K // 16):
        raise ValueError("inconsistent shapes")
    y = _out(out, (M, N), torch.bfloat16, x)
    _raise(lib.nvfp4g16_gemv_variant(x.data_ptr(), M, K, qweight.data_ptr(), scale_e4m3.data_ptr(), float(global_scale), N,
                                     y.data_ptr(), int(variant), _stream(x)))
    return y


def _nv_task_array(items):
    items = list(items)
    if not 1 <= len(items) <= 8:
        raise ValueError("1..8 tasks per call")
    arr = (NvTask * len(items))()
    outs, M = [], None
    for i, (x, qweight, scale_e4m3, global_scale, out) in enumerate(items):
        _check(x, "x", _U16, 2); _check(qweight, "qweight", _U8, 2); _check(scale_e4m3, "scale_e4m3", _E4M3, 2)
        m, K = x.shape
        N = qweight.shape[0]
        M = m if M is None else M
        if m != M:
            raise ValueError("all tasks must share the batch size M")
        if qweight.shape[1] * 2 != K or tuple(scale_e4m3.shape) != (N, K // 16):
            raise ValueError(f"task {i}: inconsistent shapes")
        y = _out(out, (M, N), torch.bfloat16, x)
        outs.append(y)
        arr[i] = NvTask(x.data_ptr(), qweight.data_ptr(), scale_e4m3.data_ptr(), float(global_scale), y.data_ptr(), N, K)
    return items, arr, outs, M


def _bf_task_array(items):
    items = list(items)
    if not 1 <= len(items) <= 8:
        raise ValueError("1..8 tasks per call")
    arr = (BfTask * len(items))()
    outs, M = [], None
    for i, (x, w, out) in enumerate(items):
        _check(x, "x", _U16, 2); _check(w, "w", _U16, 2)
        m, K = x.shape
        N = w.shape[0]
        M = m if M is None else M
        if m != M:
            raise ValueError("all tasks must share the batch size M")
        if w.shape[1] != K:
            raise ValueError(f"task {i}: inconsistent shapes")
        y = _out(out, (M, N), torch.bfloat16, x)
        outs.append(y)
        arr[i] = BfTask(x.data_ptr(), w.data_ptr(), y.data_ptr(), N, K)
    return items, arr, outs, M


def _grouped(fn, items, arr, M, variant, workspace):
    st = _stream(items[0][0])
    if workspace is None:
        _raise(fn(arr, len(items), M, int(variant), None, 0, st))
    else:
        if workspace.device != items[0][0].device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the activations' device")
        _raise(fn(arr, len(items), M, int(variant), workspace.data_ptr(), workspace.numel(), st))


def nvfp4g16_gemv_grouped(items, variant: int = VARIANT_AUTO, workspace=None):
    """Several independent NVFP4 GEMVs with one batch size, launched together.
    items: sequence of (x, qweight, scale_e4m3, global_scale, out-or-None);
    workspace as for q4g128_gemv_grouped.  Returns the list of outputs."""
    items, arr, outs, M = _nv_task_array(items)
    _grouped(lib.nvfp4g16_gemv_grouped_ws, items, arr, M, variant, workspace)
    return outs


def nvfp4g16_workspace_bytes(items) -> int:
    items, arr, _, M = _nv_task_array(items)
    n = ctypes.c_size_t(0)
    _raise(lib.nvfp4g16_workspace_bytes(arr, len(items), M, ctypes.byref(n)))
    return int(n.value)


def bf16_gemv_grouped(items, variant: int = VARIANT_AUTO, workspace=None):
    """Several independent BF16 GEMVs with one batch size, launched together.
    items: sequence of (x, w, out-or-None); workspace as for
    q4g128_gemv_grouped.  Returns the list of outputs."""
    items, arr, outs, M = _bf_task_array(items)
    _grouped(lib.bf16_gemv_grouped_ws, items, arr, M, variant, workspace)
    return outs


def bf16_workspace_bytes(items) -> int:
    items, arr, _, M = _bf_task_array(items)
    n = ctypes.c_size_t(0)
    _raise(lib.bf16_workspace_bytes(arr, len(items), M, ctypes.byref(n)))
    return int(n.value)


def bf16_gemv(x, w, out=None, variant: int = VARIANT_AUTO):
    """y[M, N] = x . W^T with W bf16 [N, K]."""
    _check(x, "x", _U16, 2); _check(w, "w", _U16, 2)
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError("inconsistent shapes")
    y = _out(out, (M, N), torch.bfloat16, x)
    _raise(lib.bf16_gemv_variant(x.data_ptr(), M, K, w.data_ptr(), N, y.data_ptr(), int(variant), _stream(x)))
    return y


def q4g128_dequant_f32(qweight, scale, minv, out=None):
    _check(qweight, "qweight", _U8, 2); _check(scale, "scale", _F16, 2); _check(minv, "min", _F16, 2)
    N, half = qweight.shape
    K = 2 * half
    w = _out(out, (N, K), torch.float32, qweight)
    _raise(lib.q4g128_dequant_f32(qweight.data_ptr(), scale.data_ptr(), minv.data_ptr(), N, K, w.data_ptr(), _stream(qweight)))
    return w


def nvfp4g16_dequant_f32(qweight, scale_e4m3, global_scale: float, out=None):
    _check(qweight, "qweight", _U8, 2); _check(scale_e4m3, "scale_e4m3", _E4M3, 2)
    N, half = qweight.shape
    K = 2 * half
    w = _out(out, (N, K), torch.float32, qweight)
    _raise(lib.nvfp4g16_dequant_f32(qweight.data_ptr(), scale_e4m3.data_ptr(), float(global_scale), N, K, w.data_ptr(),
                                    _stream(qweight)))
    return w


def _read_args(tensors):
    n = len(tensors)
    ptrs = (_p * n)(*[t.data_ptr() for t in tensors])
    sizes = (ctypes.c_size_t * n)(*[t.numel() * t.element_size() for t in tensors])
    return ptrs, sizes, n


def stream_read_sink_words(tensors) -> int:
    """Sink words stream_read needs for these device tensors (0: invalid)."""
    _, sizes, n = _read_args(tensors)
    return int(lib.q4gemv_stream_read_sink_words(sizes, n))


def stream_read(tensors, sink):
    """Diagnostic plain read of the bytes of up to 32 contiguous device tensors
    in one launch (the reference a GEMV launch of the same bytes is compared
    with); one XOR word per wave lands in the int32 device tensor `sink`."""
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("stream_read takes contiguous device tensors")
    ptrs, sizes, n = _read_args(tensors)
    _raise(lib.q4gemv_stream_read(ptrs, sizes, n, sink.data_ptr(), sink.numel(), _stream(sink)))
    return sink


def _fused_task_array(items):
    items = [dict(it) for it in items]
    if not 1 <= len(items) <= 8:
        raise ValueError("1..8 tasks per call")
    arr = (FusedTask * len(items))()
    outs, M = [], None
    for i, it in enumerate(items):
        x, qweight, scale, minv = it["x"], it["qweight"], it["scale"], it["min"]
        up, res, out = it.get("up"), it.get("residual"), it.get("out")
        _check(x, "x", _U16, 2); _check(qweight, "qweight", _U8, 2)
        _check(scale, "scale", _F16, 2); _check(minv, "min", _F16, 2)
        m, K = x.shape
        N = qweight.shape[0]
        M = m if M is None else M
        if m != M:
            raise ValueError("all tasks must share the batch size M")
        if qweight.shape[1] * 2 != K or tuple(scale.shape) != (N, K // 128) or tuple(minv.shape) != (N, K // 128):
            raise ValueError(f"task {i}: inconsistent shapes")
        if up is not None:
            _check(up, "up", _U16, 2)
            if tuple(up.shape) != (M, K):
                raise ValueError(f"task {i}: up must be [M, K]")
        if res is not None:
            _check(res, "residual", _U16, 2)
            if tuple(res.shape) != (M, N):
                raise ValueError(f"task {i}: residual must be [M, N]")
        y = _out(out, (M, N), torch.bfloat16, x)
        outs.append(y)
        arr[i] = FusedTask(x.data_ptr(), up.data_ptr() if up is not None else None, qweight.data_ptr(), scale.data_ptr(),
                           minv.data_ptr(), res.data_ptr() if res is not None else None, y.data_ptr(), N, K)
    return items, arr, outs, M


def q4g128_gemv_fused(items, workspace=None):
    """int4 g128 GEMVs with the decode step's elementwise neighbours fused
    (q4g128_gemv_fused in the C header).  items: sequence of dicts with keys
    x, qweight, scale, min and optionally up (activations become
    RN_bf16(silu(x) * up)), residual (added to the output before its
    rounding; may be the out tensor itself) and out.  workspace as for
    q4g128_gemv_grouped.  Returns the list of outputs."""
    items, arr, outs, M = _fused_task_array(items)
    st = _stream(items[0]["x"])
    if workspace is None:
        _raise(lib.q4g128_gemv_fused(arr, len(items), M, None, 0, st))
    else:
        if workspace.device != items[0]["x"].device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the activations' device")
        _raise(lib.q4g128_gemv_fused(arr, len(items), M, workspace.data_ptr(), workspace.numel(), st))
    return outs


def q4g128_fused_workspace_bytes(items) -> int:
    items, arr, _, M = _fused_task_array(items)
    n = ctypes.c_size_t(0)
    _raise(lib.q4g128_fused_workspace_bytes(arr, len(items), M, ctypes.byref(n)))
    return int(n.value)


def _sample_outputs(M, top_k, like, want_topk):
    tok = torch.empty(M, dtype=torch.int32, device=like.device)
    if not want_topk:
        return tok, None, None
    return (tok, torch.empty((M, top_k), dtype=torch.int32, device=like.device),
            torch.empty((M, top_k), dtype=torch.float32, device=like.device))


def sample_topk(logits, u, temperature: float = 0.8, top_k: int = 30, return_topk: bool = False):
    """Top-k sampling from BF16 logits [M, V] with the caller's uniforms u
    (fp32 [M], in [0, 1)): returns token int32 [M], and with return_topk also
    the top-k indices int32 [M, k] and probabilities fp32 [M, k]."""
    _check(logits, "logits", _U16, 2); _check(u, "u", (torch.float32,), 1)
    M, V = logits.shape
    if u.shape[0] != M:
        raise ValueError("u must hold one draw per batch row")
    tok, ti, tp = _sample_outputs(M, top_k, logits, return_topk)
    _raise(lib.q4_sample_topk(logits.data_ptr(), M, V, float(temperature), int(top_k), u.data_ptr(), tok.data_ptr(),
                              ti.data_ptr() if ti is not None else None, tp.data_ptr() if tp is not None else None,
                              _stream(logits)))
    return (tok, ti, tp) if return_topk else tok


def bf16_head_sample_workspace_bytes(M: int, N: int, K: int, top_k: int = 30) -> int:
    """Bytes of zero-filled workspace for the workspace head sampling (one
    launch at M = 1, the split sampler for a batch; 0 if it does not apply to
    this shape)."""
    return int(lib.bf16_head_sample_workspace_bytes(M, N, K, top_k))


def bf16_head_sample(x, w, u, temperature: float = 0.8, top_k: int = 30, logits=None, return_topk: bool = False,
                     workspace=None):
    """The BF16 head GEMV logits = x W^T followed by top-k sampling: two
    launches; with a zero-filled uint8 workspace of at least
    bf16_head_sample_workspace_bytes() (when that is nonzero),
    bf16_head_sample_ws in the C header -- one launch for one row, the split
    sampler for a batch.  Returns (token, logits) or (token, topk_index,
    topk_prob, logits) with return_topk."""
    _check(x, "x", _U16, 2); _check(w, "w", _U16, 2); _check(u, "u", (torch.float32,), 1)
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K or u.shape[0] != M:
        raise ValueError("inconsistent shapes")
    lg = _out(logits, (M, N), torch.bfloat16, x)
    tok, ti, tp = _sample_outputs(M, top_k, x, return_topk)
    ti_p = ti.data_ptr() if ti is not None else None
    tp_p = tp.data_ptr() if tp is not None else None
    if workspace is None:
        _raise(lib.bf16_head_sample(x.data_ptr(), M, K, w.data_ptr(), N, lg.data_ptr(), float(temperature), int(top_k), u.data_ptr(),
                                    tok.data_ptr(), ti_p, tp_p, _stream(x)))
    else:
        if workspace.device != x.device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the activations' device")
        _raise(lib.bf16_head_sample_ws(x.data_ptr(), M, K, w.data_ptr(), N, lg.data_ptr(), float(temperature), int(top_k),
                                       u.data_ptr(), tok.data_ptr(), ti_p, tp_p, workspace.data_ptr(), workspace.numel(), _stream(x)))
    return (tok, ti, tp, lg) if return_topk else (tok, lg)


def q4g128_gemm(x, qweight, scale, minv, out=None, variant: int = VARIANT_AUTO):
    """Prefill GEMM y[M, N] = x[M, K] . W^T for int4 g128 weights, any M
    (q4g128_gemm_variant in the C header: VARIANT_AUTO, VARIANT_TILED for the
    tiled decode kernel over batch chunks, VARIANT_GEMM for the large-tile
    prefill kernel)."""
    _check(x, "x", _U16, 2); _check(qweight, "qweight", _U8, 2)
    _check(scale, "scale", _F16, 2); _check(minv, "min", _F16, 2)
    M, K = x.shape
    N = qweight.shape[0]
    if qweight.shape[1] * 2 != K or tuple(scale.shape) != (N, K // 128) or tuple(minv.shape) != (N, K // 128):
        raise ValueError("inconsistent shapes")
    y = _out(out, (M, N), torch.bfloat16, x)
    _raise(lib.q4g128_gemm_variant(x.data_ptr(), M, K, qweight.data_ptr(), scale.data_ptr(), minv.data_ptr(), N, y.data_ptr(),
                                   variant, _stream(x)))
    return y


def _mixed_task_array(items):
    """Tagged task tuples -> (MixedTask array, outputs, M):
      ("q4g128", x, qweight, scale, min, out), ("nvfp4g16", x, qweight,
      scale_e4m3, global_scale, out), ("bf16", x, w, out); out may be None."""
    items = list(items)
    if not 1 <= len(items) <= 8:
        raise ValueError("1..8 tasks per call")
    arr = (MixedTask * len(items))()
    outs, M = [], None
    for i, it in enumerate(items):
        kind = it[0]
        if kind == "q4g128":
            _, x, qw, sc, mn, out = it
            _check(qw, "qweight", _U8, 2); _check(sc, "scale", _F16, 2); _check(mn, "min", _F16, 2)
            fmt, w, G, N, K = FMT_Q4G128, qw, 0.0, qw.shape[0], qw.shape[1] * 2
            if tuple(sc.shape) != (N, K // 128) or tuple(mn.shape) != (N, K // 128):
                raise ValueError(f"task {i}: inconsistent shapes")
        elif kind == "nvfp4g16":
            _, x, qw, sc, G, out = it
            _check(qw, "qweight", _U8, 2); _check(sc, "scale_e4m3", _E4M3, 2)
            fmt, w, mn, N, K = FMT_NVFP4G16, qw, None, qw.shape[0], qw.shape[1] * 2
            if tuple(sc.shape) != (N, K // 16):
                raise ValueError(f"task {i}: inconsistent shapes")
        elif kind == "bf16":
            _, x, w, out = it
            _check(w, "w", _U16, 2)
            fmt, sc, mn, G, (N, K) = FMT_BF16, None, None, 0.0, w.shape
        else:
            raise ValueError(f"unknown task kind {kind!r} (q4g128, nvfp4g16, bf16)")
        _check(x, "x", _U16, 2)
        if x.shape[1] != K:
            raise ValueError(f"task {i}: x has K = {x.shape[1]}, the weights {K}")
        M = x.shape[0] if M is None else M
        if x.shape[0] != M:
            raise ValueError("all tasks must share the batch size M")
        y = _out(out, (M, N), torch.bfloat16, x)
        outs.append(y)
        arr[i] = MixedTask(fmt, x.data_ptr(), w.data_ptr(), sc.data_ptr() if sc is not None else None,
                           mn.data_ptr() if mn is not None else None, float(G), y.data_ptr(), N, K)
    return items, arr, outs, M


def gemv_grouped_mixed(items, workspace=None):
    """Independent GEMVs of mixed weight formats with one batch size, in one
    launch where the streaming kernel takes them all (M <= 4), else one
    grouped launch per format (q4gemv_grouped_mixed in the C header).
    Returns the list of outputs."""
    items, arr, outs, M = _mixed_task_array(items)
    st = _stream(items[0][1])
    if workspace is None:
        _raise(lib.q4gemv_grouped_mixed(arr, len(items), M, None, 0, st))
    else:
        if workspace.device != items[0][1].device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the activations' device")
        _raise(lib.q4gemv_grouped_mixed(arr, len(items), M, workspace.data_ptr(), workspace.numel(), st))
    return outs


def mixed_workspace_bytes(items) -> int:
    items, arr, _, M = _mixed_task_array(items)
    n = ctypes.c_size_t(0)
    _raise(lib.q4gemv_mixed_workspace_bytes(arr, len(items), M, ctypes.byref(n)))
    return int(n.value)


# ---------------------------------------------------------------------------
# 8-bit block-scaled products and the verification of drafted tokens.  These
# calls may be made while another device than the tensors' is current.
# ---------------------------------------------------------------------------
_F32, _I32, _BF16 = (torch.float32,), (torch.int32,), (torch.bfloat16,)
_BLOCK = 128
_FP8_TASK = struct.Struct("6Q2i").pack      # an Fp8Task's bytes (a tenth of the structure's own construction)
assert ctypes.sizeof(Fp8Task) == 56
# the raw handle of the current stream; building a Stream object costs as much
# as a launch
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _refuse(t, name: str, dtypes, shape, index: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    raise ValueError(f"{name} must be contiguous")


def _tensor(t, name: str, dtypes, shape, index: int) -> int:
    """Address of a contiguous tensor of this shape on GPU `index`, or an error
    that names what is wrong."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        return t.data_ptr()
    _refuse(t, name, dtypes, shape, index)


def _optional(t, name: str, dtypes, shape, index: int):
    return None if t is None else _tensor(t, name, dtypes, shape, index)


def _scratch(workspace, index: int):
    if workspace is None:
        return None, 0
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.dtype != torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return workspace.data_ptr(), workspace.numel()


def _enqueue(index: int, fn, *args):
    """fn(*args, stream) on GPU index's current stream, with that GPU current (a
    launch goes to the current device)."""
    if _get_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != 0:
        raise Q4GemvError(rc)


def fp8b128_quantize(x, up=None, codes=None, scale=None):
    """e4m3 codes [M, K] (torch.float8_e4m3fn) and fp32 scales
    [M, ceil(K / 128)] of bf16 activations x, or of silu(x) * up; K a multiple
    of 16.  codes and scale: outputs to write into.  Returns (codes, scale)."""
    _check(x, "x", _U16, 2)
    shape, index = x.shape, x.get_device()
    M, K = shape
    G = (K + _BLOCK - 1) // _BLOCK
    up_p = None if up is None else _tensor(up, "up", _U16, shape, index)
    if codes is None:
        codes = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        codes_p = codes.data_ptr()
    else:
        codes_p = _tensor(codes, "codes", _E4M3, shape, index)
    if scale is None:
        scale = x.new_empty((M, G), dtype=torch.float32)
        scale_p = scale.data_ptr()
    else:
        scale_p = _tensor(scale, "scale", _F32, (M, G), index)
    _enqueue(index, lib.fp8b128_quantize, x.data_ptr(), up_p, M, K, codes_p, scale_p)
    return codes, scale


_NO_OUTPUT = 1 << 60      # an address that no tensor has, and room for any output behind it


def _fp8_task_array(items, sizing=False):
    """The tasks' bytes, their count, the outputs, M and the device.  sizing: for
    a question about sizes alone, outputs that are not given are not made."""
    items = list(items)
    count = len(items)
    if not 1 <= count <= 8:
        raise ValueError("1..8 tasks per call")
    arr, outs, M, index = [], [], None, None
    last, last_scale = None, None
    for x, x_scale, w, w_scale, residual, out in items:
        if x is not last or x_scale is not last_scale:
            _check(x, "x", _E4M3, 2)
            m, K = x.shape
            if M is None:
                M, index = m, x.get_device()
            elif m != M or x.get_device() != index:
                raise ValueError("all tasks must share the batch size M and the device")
            G = (K + _BLOCK - 1) // _BLOCK
            xp, sp = x.data_ptr(), _tensor(x_scale, "x_scale", _F32, (M, G), index)
            last, last_scale = x, x_scale
        if not isinstance(w, torch.Tensor) or w.dim() != 2:
            raise ValueError("w must be a tensor of 2 dims")
        N = w.shape[0]
        if out is not None:
            y, yp = out, _tensor(out, "out", _BF16, (M, N), index)
        elif sizing:
            y, yp = None, _NO_OUTPUT + (len(arr) << 50)
        else:
            y = x_scale.new_empty((M, N), dtype=torch.bfloat16)
            yp = y.data_ptr()
        outs.append(y)
        arr.append(_FP8_TASK(xp, sp, _tensor(w, "w", _E4M3, (N, K), index),
                             _tensor(w_scale, "w_scale", _F32, ((N + _BLOCK - 1) // _BLOCK, G), index),
                             0 if residual is None else _tensor(residual, "residual", _U16, (M, N), index),
                             yp, N, K))
    return b"".join(arr), count, outs, M, index


def fp8b128_gemm_grouped(items, workspace=None):
    """Several independent 8-bit block-scaled products with one batch size,
    launched together.  items: sequence of (x, x_scale, w, w_scale,
    residual-or-None, out-or-None): x e4m3 [M, K] with x_scale fp32
    [M, ceil(K / 128)] (fp8b128_quantize makes both), w e4m3 [N, K] with
    w_scale fp32 [ceil(N / 128), ceil(K / 128)], residual and out bf16 [M, N]
    (out may be the residual).  workspace: optional uint8 device tensor of at
    least fp8b128_workspace_bytes(items) bytes, zero-filled before its first
    use and reusable afterwards without clearing (lets few rows split K; a
    smaller one lets them less).
    Returns the list of outputs."""
    arr, count, outs, M, index = _fp8_task_array(items)
    _enqueue(index, lib.fp8b128_gemm_grouped_ws, arr, count, M, *_scratch(workspace, index))
    return outs


def fp8b128_workspace_bytes(items) -> int:
    """Bytes of workspace fp8b128_gemm_grouped can use for these items (0: none)."""
    arr, count, _, M, _ = _fp8_task_array(items, sizing=True)
    n = ctypes.c_size_t(0)
    _raise(lib.fp8b128_workspace_bytes(arr, count, M, ctypes.byref(n)))
    return int(n.value)


def fp8b128_gemm(x, x_scale, w, w_scale, residual=None, out=None, workspace=None):
    """y[M, N] = sum over blocks of 128 columns of x_scale * w_scale * (x . W^T)
    (+ residual), bf16: one product of fp8b128_gemm_grouped."""
    return fp8b128_gemm_grouped(((x, x_scale, w, w_scale, residual, out),), workspace)[0]


def verify_topk_workspace_bytes(B: int, D: int, V: int, top_k: int = 30) -> int:
    """Bytes of workspace verify_topk uses (0: none)."""
    return int(lib.q4_verify_topk_workspace_bytes(B, D, V, top_k))


def verify_full_workspace_bytes(B: int, D: int, V: int) -> int:
    """Bytes of workspace verify_full uses."""
    return int(lib.q4_verify_full_workspace_bytes(B, D, V))


def verify_topk(logits, draft, u, draft_index=None, draft_prob=None, n_draft=None, temperature: float = 0.8, top_k: int = 30,
                workspace=None):
    """Verifies drafted tokens against the target's top-k distributions
    (q4_verify_topk in the C header): logits bf16 [B, D + 1, V], draft int32
    [B, D], u fp32 [B, D + 1] in [0, 1) (D acceptance uniforms, then the
    draw's), the draft's distributions as draft_index int32 and draft_prob fp32
    [B, D, k'] (sample_topk's outputs) or None for a draft certain of its
    tokens, n_draft int32 [B] or None.  workspace: uint8, at least
    verify_topk_workspace_bytes, zero-filled before its first use and reusable
    afterwards without clearing (None: one is made for the call).
    Returns (token int32 [B, D + 1]: the tokens that stand, the one drawn after
    them, then -1; count int32 [B]: how many stand; accept_prob fp32 [B, D])."""
    _check(logits, "logits", _U16, 3)
    B, D1, V = logits.shape
    D, index = D1 - 1, logits.get_device()
    if workspace is None:
        workspace = logits.new_empty(verify_topk_workspace_bytes(B, D, V, top_k), dtype=torch.uint8)
    kd = 0
    if draft_index is not None:
        if not isinstance(draft_index, torch.Tensor) or draft_index.dim() != 3:
            raise ValueError("draft_index must be a tensor of 3 dims")
        kd = draft_index.shape[2]
    up, dp = _tensor(u, "u", _F32, (B, D1), index), _tensor(draft, "draft", _I32, (B, D), index)
    token = torch.empty_like(u, dtype=torch.int32)
    count = u.new_empty(B, dtype=torch.int32)
    prob = torch.empty_like(draft, dtype=torch.float32)
    _enqueue(index, lib.q4_verify_topk, logits.data_ptr(), B, D, V, dp,
             _optional(draft_index, "draft_index", _I32, (B, D, kd), index),
             _optional(draft_prob, "draft_prob", _F32, (B, D, kd), index), kd, _optional(n_draft, "n_draft", _I32, (B,), index),
             up, temperature, top_k, token.data_ptr(), count.data_ptr(), prob.data_ptr(),
             *_scratch(workspace, index))
    return token, count, prob


def verify_full(logits, draft, u, draft_logits=None, n_draft=None, temperature: float = 0.8, workspace=None):
    """Verifies drafted tokens against the softmax of whole rows
    (q4_verify_full in the C header): as verify_topk, with the draft's
    distributions as draft_logits bf16 [B, D, V] or None."""
    _check(logits, "logits", _U16, 3)
    B, D1, V = logits.shape
    D, index = D1 - 1, logits.get_device()
    if workspace is None:
        workspace = logits.new_zeros(verify_full_workspace_bytes(B, D, V), dtype=torch.uint8)
    up, dp = _tensor(u, "u", _F32, (B, D1), index), _tensor(draft, "draft", _I32, (B, D), index)
    token = torch.empty_like(u, dtype=torch.int32)
    count = u.new_empty(B, dtype=torch.int32)
    prob = torch.empty_like(draft, dtype=torch.float32)
    _enqueue(index, lib.q4_verify_full, logits.data_ptr(), B, D, V, dp,
             _optional(draft_logits, "draft_logits", _U16, (B, D, V), index), _optional(n_draft, "n_draft", _I32, (B,), index),
             up, temperature, token.data_ptr(), count.data_ptr(), prob.data_ptr(),
             *_scratch(workspace, index))
    return token, count, prob


# ---------------------------------------------------------------------------
# A decoder layer's attention.  As above, another device may be current.
# ---------------------------------------------------------------------------
class KvCache(ctypes.Structure):
    """Mirror of the C struct q4_kv_cache (an object of it, or its bytes)."""
    _fields_ = [("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p), ("pages", _i), ("page_size", _i)]


_KV_CACHE = struct.Struct("4Q2i").pack      # a KvCache's bytes
assert ctypes.sizeof(KvCache) == 40
_SLOT = (torch.int64,)


def _heads(t, name: str, index: int, tokens=None, heads=None, D=None) -> int:
    """Elements from a token of bf16 heads [tokens, heads, D] to the next; a
    token's heads follow each other."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _U16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {_U16}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dims, got shape {tuple(t.shape)}")
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name} is on {t.device}, expected " + (f"cuda:{index}" if index >= 0 else "a GPU"))
    n, h, d = t.shape
    if (tokens is not None and n != tokens) or (heads is not None and h != heads) or (D is not None and d != D):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(tokens or n, heads or h, D or d)}")
    stride, of_head, one = t.stride()
    if one != 1 or (of_head != d and h > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return stride if n > 1 else h * d


def _kv_cache(cache, index: int, Hk: int, D: int):
    """The C struct's bytes of (k, v) or (k, v, k_scale, v_scale), and the page size."""
    cache = tuple(cache)
    if len(cache) not in (2, 4):
        raise ValueError("cache must be (k, v) or (k, v, k_scale, v_scale)")
    k, v = cache[:2]
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or k.shape[1] != Hk or k.shape[3] != D:
        raise ValueError(f"cache: k must be a tensor [pages, {Hk}, page_size, {D}]")
    pages, _, page_size, _ = k.shape
    types = _E4M3 if len(cache) == 4 else _U16
    kp, vp = _tensor(k, "cache: k", types, k.shape, index), _tensor(v, "cache: v", types, k.shape, index)
    ksp = vsp = 0
    if len(cache) == 4:
        shape = (pages, Hk, page_size)
        ksp, vsp = _tensor(cache[2], "cache: k_scale", _F32, shape, index), _tensor(cache[3], "cache: v_scale", _F32, shape, index)
    return _KV_CACHE(kp, vp, ksp, vsp, pages, page_size), page_size


def _rotated(out, name: str, shape, index: int, x, stride: int):
    """A contiguous output for the heads x.  The library takes an output at x's
    address for x itself, its tokens `stride` elements apart."""
    if _tensor(out, name, _U16, shape, index) == x.data_ptr() and stride != shape[1] * shape[2]:
        raise ValueError(f"{name} begins where {name[0]} does, whose tokens lie apart: in place is {name[0]} itself")


def rope_cache(q, k, v=None, positions=None, inv_freq=None, q_norm=None, k_norm=None, eps: float = 1e-6, interleaved: bool = False,
               cache=None, slots=None, q_out=None, k_out=None):
    """q's and k's heads normalised (q_norm, k_norm: bf16 weights [D], or None)
    and rotated (positions int32 [T], inv_freq fp32 [rot / 2], None: no
    rotation), and k and v appended to a paged cache (q4_rope_cache in the C
    header).  q bf16 [T, Hq, D], k and v [T, Hk, D]; their tokens may lie
    apart, as parts of one product's rows do.  cache: (k, v) bf16
    [pages, Hk, page_size, D], or (k, v, k_scale, v_scale) with e4m3 codes and
    fp32 scales [pages, Hk, page_size]; slots int64 [T]: page * page_size +
    place of each token, -1 to not keep it.  q_out: a tensor to write into (q
    itself: in place); k_out the same, True for a new one, None for none (a new
    one without a cache).  Returns (q_out, k_out)."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    index = q.get_device()
    qs = _heads(q, "q", index)
    T, Hq, D = q.shape
    ks = _heads(k, "k", index, T, None, D)
    Hk = k.shape[1]
    vs, rot, vp, sp, cp = Hk * D, 0, None, None, None
    if cache is not None:
        vs, vp = _heads(v, "v", index, T, Hk, D), v.data_ptr()
        sp = _tensor(slots, "slots", _SLOT, (T,), index)
        cp, _ = _kv_cache(cache, index, Hk, D)
    elif v is not None or slots is not None:
        raise ValueError("v and slots are of a cache, and there is none")
    pp = fp = None
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be a tensor of 1 dim")
        rot = 2 * inv_freq.shape[0]
        fp, pp = _tensor(inv_freq, "inv_freq", _F32, inv_freq.shape, index), _tensor(positions, "positions", _I32, (T,), index)
    if q_out is None:
        q_out = q.new_empty((T, Hq, D))
    elif q_out is not q:
        _rotated(q_out, "q_out", (T, Hq, D), index, q, qs)
    if k_out is True or (k_out is None and cache is None):
        k_out = k.new_empty((T, Hk, D))
    elif k_out is not None and k_out is not k:
        _rotated(k_out, "k_out", (T, Hk, D), index, k, ks)
    _enqueue(index, lib.q4_rope_cache, q.data_ptr(), k.data_ptr(), vp, T, Hq, Hk, D, qs, ks, vs,
             _optional(q_norm, "q_norm", _U16, (D,), index), _optional(k_norm, "k_norm", _U16, (D,), index), eps, pp, fp, rot,
             1 if interleaved else 0, q_out.data_ptr(), None if k_out is None else k_out.data_ptr(), cp, sp)
    return q_out, k_out


def _window(window):
    if not -2 ** 31 <= window < 2 ** 31:
        raise ValueError("window must be below 2^31")
    return window


def attention_decode_workspace_bytes(T: int, Hq: int, Hk: int, D: int) -> int:
    """Bytes of workspace attention_decode uses for T new tokens a sequence."""
    return int(lib.q4_attention_decode_workspace_bytes(T, Hq, Hk, D))


def attention_decode(q, cache, table, lengths, n_new=None, scale=None, window: int = 0, out=None, workspace=None):
    """Attention of new tokens over a paged cache that already holds them
    (q4_attention_decode in the C header): q bf16 [B, T, Hq, D], cache as for
    rope_cache, table int32 [B, width] of page numbers (-1: none), lengths int32
    [B] with the new tokens, n_new int32 [B] (None: T each), scale (None:
    D ** -0.5), window (0: all keys).  workspace: uint8, at least
    attention_decode_workspace_bytes, zero-filled before its first use and
    reusable afterwards without clearing (None: one is made and cleared for the
    call, 2 to 17 MiB, which adds 3 to 5 us to it).
    Returns bf16 [B, T, Hq, D]; rows that see no key are 0."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.dim() != 4:
        raise ValueError(f"q must have 4 dims, got shape {tuple(q.shape)}")
    index = q.get_device()
    B, T, Hq, D = q.shape
    if q.is_contiguous():
        if index < 0 or q.dtype not in _U16:
            _heads(q.view(B * T, Hq, D), "q", index)
        stride = Hq * D
    else:
        if B > 1 and T > 1 and q.stride(0) != T * q.stride(1):
            raise ValueError("q: rows of all tokens must lie equally far apart")
        stride = _heads(q[:, 0] if T == 1 else q[0] if B == 1 else q.flatten(0, 1), "q", index)
    if not isinstance(cache[0], torch.Tensor) or cache[0].dim() != 4:
        raise ValueError("cache: k must be a tensor of 4 dims")
    Hk = cache[0].shape[1]
    cp, _ = _kv_cache(cache, index, Hk, D)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a tensor of 2 dims")
    width = table.shape[1]
    tp, lp = _tensor(table, "table", _I32, (B, width), index), _tensor(lengths, "lengths", _I32, (B,), index)
    if workspace is None:
        workspace = q.new_zeros(attention_decode_workspace_bytes(T, Hq, Hk, D), dtype=torch.uint8)
    if out is None:
        out = q.new_empty((B, T, Hq, D))
    else:
        _tensor(out, "out", _U16, (B, T, Hq, D), index)
    _enqueue(index, lib.q4_attention_decode, q.data_ptr(), B, T, Hq, Hk, D, stride, cp, tp, width, lp,
             _optional(n_new, "n_new", _I32, (B,), index), D ** -0.5 if scale is None else scale, _window(window), out.data_ptr(),
             *_scratch(workspace, index))
    return out


def attention_prefill(q, k, v, starts, key_starts=None, scale=None, window: int = 0, out=None):
    """Causal attention over packed prompts (q4_attention_prefill in the C
    header): q bf16 [T, Hq, D], k and v [S, Hk, D] (tokens may lie apart),
    sequence b's tokens rows starts[b] .. starts[b + 1] of q, its keys rows
    key_starts[b] .. key_starts[b + 1] of k and v (None: starts, S = T); int32
    [B + 1].  The last token sees the last key.  scale and window as for
    attention_decode.  Returns bf16 [T, Hq, D]; rows of no sequence are not
    written."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    index = q.get_device()
    qs = _heads(q, "q", index)
    T, Hq, D = q.shape
    ks = _heads(k, "k", index, T if key_starts is None else None, None, D)
    S, Hk, _ = k.shape
    vs = _heads(v, "v", index, S, Hk, D)
    if not isinstance(starts, torch.Tensor) or starts.dim() != 1:
        raise ValueError("starts must be a tensor of 1 dim")
    n = starts.shape[0]
    sp, kp = _tensor(starts, "starts", _I32, (n,), index), _optional(key_starts, "key_starts", _I32, (n,), index)
    if out is None:
        out = q.new_empty((T, Hq, D))
    else:
        _tensor(out, "out", _U16, (T, Hq, D), index)
    _enqueue(index, lib.q4_attention_prefill, q.data_ptr(), T, k.data_ptr(), v.data_ptr(), S, Hq, Hk, D, qs, ks, vs, sp, kp, n - 1,
             D ** -0.5 if scale is None else scale, _window(window), out.data_ptr())
    return out
