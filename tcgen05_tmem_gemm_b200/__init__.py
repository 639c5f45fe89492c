"""Python binding of libdg, the B200 (sm_100a) strided-view GEMM library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in include/dg.h.  The names mirror the C
entry points (dg_gemm, dg_gemm_ex, dg_gemv, dg_sync_status, ...).  PyTorch is used by
callers for device memory and streams; a torch tensor can be turned into a
view with `view()`.

The library must have been built (``python tcgen05_tmem_gemm_b200/build.py``
or ``__graft_entry__.build()``); importing this package without it raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")

DG_F32, DG_F16, DG_BF16, DG_E4M3 = 0, 1, 2, 3
DTYPE = {"f32": DG_F32, "f16": DG_F16, "bf16": DG_BF16, "e4m3": DG_E4M3}
ELEM_SIZE = {DG_F32: 4, DG_F16: 2, DG_BF16: 2, DG_E4M3: 1}

(DG_OK, DG_ERR_NULL, DG_ERR_NDIM, DG_ERR_SHAPE, DG_ERR_DTYPE, DG_ERR_STRIDE, DG_ERR_ALIGN,
 DG_ERR_POINTER, DG_ERR_VALUE, DG_ERR_UNSUPPORTED, DG_ERR_CUDA, DG_ERR_TIMEOUT) = range(12)

(DG_KIND_NONE, DG_KIND_SCALE_C, DG_KIND_SIMT, DG_KIND_GEMV_N, DG_KIND_GEMV_K,
 DG_KIND_UMMA) = range(6)
KIND_NAME = {0: "none", 1: "scale_c", 2: "simt", 3: "gemv_n", 4: "gemv_k", 5: "umma"}

DG_ACT_NONE, DG_ACT_RELU, DG_ACT_GELU_TANH = 0, 1, 2
ACT = {"none": DG_ACT_NONE, "relu": DG_ACT_RELU, "gelu_tanh": DG_ACT_GELU_TANH}

(DG_OPT_FORCE_KIND, DG_OPT_WAIT_TIMEOUT_MS, DG_OPT_TEST_STALL, DG_OPT_MAX_SPLIT_K, DG_OPT_CTA_PAIR,
 DG_OPT_EARLY_LAUNCH, DG_OPT_TRACE, DG_OPT_EPI_TMA, DG_OPT_GATHER_CLUSTER,
 DG_OPT_PAIR_TAIL, DG_OPT_STREAM_K, DG_OPT_DETERMINISTIC,
 DG_OPT_PAIR_DEEP_STAGES) = 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13


class dg_view(ctypes.Structure):
    _fields_ = [
        ("ptr", ctypes.c_void_p),
        ("ndim", ctypes.c_int32),
        ("row_dims", ctypes.c_int32),
        ("shape", ctypes.c_int64 * 4),
        ("stride", ctypes.c_int64 * 4),
        ("dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class dg_epilogue(ctypes.Structure):
    _fields_ = [
        ("bias", ctypes.c_void_p),
        ("activation", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class dg_view_info(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
        ("n_row", ctypes.c_int32), ("n_col", ctypes.c_int32),
        ("row_shape", ctypes.c_int64 * 4), ("row_stride", ctypes.c_int64 * 4),
        ("col_shape", ctypes.c_int64 * 4), ("col_stride", ctypes.c_int64 * 4),
        ("unit_dim", ctypes.c_int32), ("tma_ok", ctypes.c_int32),
        ("span_bytes", ctypes.c_int64),
        ("vec_bytes", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class dg_plan_info(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32), ("swap_ab", ctypes.c_int32), ("p_gather", ctypes.c_int32),
        ("p_mn_major", ctypes.c_int32), ("q_mn_major", ctypes.c_int32),
        ("block_m", ctypes.c_int32), ("block_n", ctypes.c_int32), ("block_k", ctypes.c_int32),
        ("stages", ctypes.c_int32), ("split_k", ctypes.c_int32), ("grid", ctypes.c_int32),
        ("vec_bytes", ctypes.c_int32),
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("cta_pair", ctypes.c_int32), ("epi_tma_store", ctypes.c_int32),
        ("gather_cluster", ctypes.c_int32), ("pair_half_tiles", ctypes.c_int32),
        ("stream_k_tiles", ctypes.c_int32), ("split_reduce_add", ctypes.c_int32),
    ]

    def as_dict(self) -> dict:
        d = {name: getattr(self, name) for name, _ in self._fields_}
        d["kind_name"] = KIND_NAME.get(self.kind, "?")
        return d


class dg_tune_result(ctypes.Structure):
    _fields_ = [
        ("candidates", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("default_us", ctypes.c_float), ("best_us", ctypes.c_float),
        ("plan", dg_plan_info),
    ]


class dg_w4(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
        ("K", ctypes.c_int64), ("N", ctypes.c_int64),
        ("code_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64), ("zero_stride", ctypes.c_int64),
        ("group", ctypes.c_int32), ("scale_dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 2),
    ]


class dg_mx4(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("scale", ctypes.c_void_p),
        ("rows", ctypes.c_int64), ("K", ctypes.c_int64), ("code_stride", ctypes.c_int64),
        ("block", ctypes.c_int32), ("reserved", ctypes.c_int32),
    ]


class DgError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libdg.so is not built ({LIB_PATH}); run python tcgen05_tmem_gemm_b200/build.py")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    V = P(dg_view)
    L.dg_gemm.argtypes = [V, V, V, ctypes.c_float, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                          ctypes.c_void_p]
    L.dg_gemm.restype = ctypes.c_int
    L.dg_gemm_ex.argtypes = [V, V, V, ctypes.c_float, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                             P(dg_epilogue), ctypes.c_void_p]
    L.dg_gemm_ex.restype = ctypes.c_int
    L.dg_gemv.argtypes = [V, V, V, ctypes.c_float, ctypes.c_float, ctypes.c_void_p]
    L.dg_gemv.restype = ctypes.c_int
    L.dg_gemv_w4.argtypes = [V, P(dg_w4), V, ctypes.c_float, ctypes.c_float, P(dg_epilogue), ctypes.c_void_p]
    L.dg_gemv_w4.restype = ctypes.c_int
    I64 = ctypes.c_int64
    L.dg_linear_ce.argtypes = [V, V, ctypes.c_void_p, I64, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                               ctypes.c_void_p, I64, ctypes.c_void_p]
    L.dg_linear_ce.restype = ctypes.c_int
    L.dg_linear_ce_grad.argtypes = [V, V, ctypes.c_void_p, I64, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, I64,
                                    V, V, ctypes.c_void_p, I64, ctypes.c_void_p]
    L.dg_linear_ce_grad.restype = ctypes.c_int
    L.dg_linear_ce_workspace.argtypes = [V, V, P(I64), P(I64)]
    L.dg_linear_ce_workspace.restype = ctypes.c_int
    L.dg_linear_ce_grad_workspace.argtypes = [V, V, V, V, P(I64), P(I64)]
    L.dg_linear_ce_grad_workspace.restype = ctypes.c_int
    I32, F = ctypes.c_int32, ctypes.c_float
    A = ctypes.c_void_p  # a structure by address: byref() or packed bytes
    L.dg_gemm_grouped.argtypes = [A, A, A, ctypes.c_void_p, I32, F, F, ctypes.c_void_p, ctypes.c_void_p,
                                  P(dg_epilogue), ctypes.c_void_p]
    L.dg_gemm_grouped.restype = ctypes.c_int
    L.dg_gemm_grouped_dw.argtypes = [A, A, A, ctypes.c_void_p, I32, F, F, ctypes.c_void_p]
    L.dg_gemm_grouped_dw.restype = ctypes.c_int
    L.dg_mx4_scale_bytes.argtypes = [I64, I64, I32]
    L.dg_mx4_scale_bytes.restype = I64
    L.dg_quantize_mx4.argtypes = [A, A, ctypes.c_void_p]
    L.dg_quantize_mx4.restype = ctypes.c_int
    L.dg_dequantize_mx4.argtypes = [A, A, ctypes.c_void_p]
    L.dg_dequantize_mx4.restype = ctypes.c_int
    L.dg_gemm_mx4.argtypes = [A, A, A, F, F, P(dg_epilogue), ctypes.c_void_p]
    L.dg_gemm_mx4.restype = ctypes.c_int
    L.dg_status_string.argtypes = [ctypes.c_int]
    L.dg_status_string.restype = ctypes.c_char_p
    L.dg_sync_status.argtypes = [ctypes.c_void_p]
    L.dg_sync_status.restype = ctypes.c_int
    L.dg_analyse_view.argtypes = [V, P(dg_view_info)]
    L.dg_analyse_view.restype = ctypes.c_int
    L.dg_plan.argtypes = [V, V, V, ctypes.c_float, ctypes.c_float, ctypes.c_int, ctypes.c_int,
                          P(dg_plan_info)]
    L.dg_plan.restype = ctypes.c_int
    L.dg_autotune.argtypes = [V, V, V, ctypes.c_float, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                              P(dg_epilogue), ctypes.c_void_p, ctypes.c_int, P(dg_tune_result)]
    L.dg_autotune.restype = ctypes.c_int
    L.dg_gemm_static.argtypes = [V, V, V, ctypes.c_float, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                 ctypes.c_void_p]
    L.dg_gemm_static.restype = ctypes.c_int
    L.dg_tune_clear.argtypes = []
    L.dg_tune_clear.restype = ctypes.c_int
    L.dg_launch_count.argtypes = []
    L.dg_launch_count.restype = ctypes.c_uint64
    L.dg_set_option.argtypes = [ctypes.c_int, ctypes.c_int64]
    L.dg_set_option.restype = ctypes.c_int
    L.dg_version.argtypes = []
    L.dg_version.restype = ctypes.c_int
    return L


lib = _load()


# ------------------------------------------------------------------ views

# dg_view, dg_w4 and dg_mx4 as packed bytes: filling a ctypes structure field by field
# costs several times as much, and small products are bound by the call.
_VIEW = struct.Struct("=Qii8qiI")
_W4 = struct.Struct("=3Q5q2i2i")
_MX4 = struct.Struct("=3Q3q2i")
assert _VIEW.size == ctypes.sizeof(dg_view) and _W4.size == ctypes.sizeof(dg_w4) and _MX4.size == ctypes.sizeof(dg_mx4)


def make_view(ptr: int, shape, stride_bytes, row_dims: int, dtype) -> dg_view:
    """A dg_view from a raw device address, up to 4 dims, BYTE strides."""
    if isinstance(dtype, str):
        dtype = DTYPE[dtype]
    v = dg_view()
    v.ptr = ctypes.c_void_p(int(ptr))
    v.ndim = len(shape)
    v.row_dims = int(row_dims)
    for i in range(4):
        v.shape[i] = int(shape[i]) if i < len(shape) else 1
        v.stride[i] = int(stride_bytes[i]) if i < len(shape) else 0
    v.dtype = int(dtype)
    v.reserved = 0
    return v


_TORCH_DT = None


def _torch_dtype_code(t) -> int:
    global _TORCH_DT
    if _TORCH_DT is None:
        import torch

        _TORCH_DT = {torch.float32: DG_F32, torch.float16: DG_F16, torch.bfloat16: DG_BF16,
                     torch.float8_e4m3fn: DG_E4M3}
    code = _TORCH_DT.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported tensor dtype {t.dtype}")
    return code


def view(t, row_dims: int = 1) -> dg_view:
    """A dg_view of a torch tensor in place (its strides, in bytes, as they are)."""
    return dg_view.from_buffer_copy(_packed_view(t, row_dims))


def _packed_view(t, row_dims: int) -> bytes:
    code = _torch_dtype_code(t)
    es = ELEM_SIZE[code]
    shape, stride = t.shape, t.stride()
    n = len(shape)
    if n == 2:
        return _VIEW.pack(t.data_ptr(), 2, row_dims, shape[0], shape[1], 1, 1, stride[0] * es, stride[1] * es, 0, 0,
                          code, 0)
    if n == 3:
        return _VIEW.pack(t.data_ptr(), 3, row_dims, *shape, 1, stride[0] * es, stride[1] * es, stride[2] * es, 0,
                          code, 0)
    if n > 4:
        raise ValueError("views have at most 4 dims")
    if n == 0:
        shape, stride = (1,), (1,)
    return bytes(make_view(t.data_ptr(), shape, [s * es for s in stride], row_dims, code))


def _as_view(x, row_dims=1):
    return x if isinstance(x, dg_view) else view(x, row_dims)


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = None


def _current_stream():
    """The current stream's handle, without the cost of a torch.cuda.Stream object where torch offers it."""
    global _raw_stream
    if _raw_stream is None:
        import torch

        raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
        _raw_stream = (lambda: raw(device())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def _stream_ptr(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# --------------------------------------------------------------- entry points

def status_string(status: int) -> str:
    return lib.dg_status_string(int(status)).decode()


def dg_gemm(A: dg_view, B: dg_view, C: dg_view, alpha: float, beta: float,
            scale_a=None, scale_b=None, stream=None) -> int:
    """C = alpha * diag(scale_a) A B diag(scale_b) + beta * C on `stream`; returns the status."""
    return lib.dg_gemm(ctypes.byref(A), ctypes.byref(B), ctypes.byref(C), float(alpha), float(beta),
                       _ptr(scale_a), _ptr(scale_b), _stream_ptr(stream))


def epilogue(bias=None, act="none") -> dg_epilogue:
    """A dg_epilogue: bias (device float32[N] tensor, address or None) and activation."""
    e = dg_epilogue()
    e.bias = ctypes.c_void_p(_ptr(bias) or 0)
    e.activation = ACT[act] if isinstance(act, str) else int(act)
    e.reserved = 0
    return e


def dg_gemm_ex(A: dg_view, B: dg_view, C: dg_view, alpha: float, beta: float,
               scale_a=None, scale_b=None, epi=None, stream=None) -> int:
    """dg_gemm with a fused epilogue C = act(... + beta * C + bias); returns the status."""
    return lib.dg_gemm_ex(ctypes.byref(A), ctypes.byref(B), ctypes.byref(C), float(alpha), float(beta),
                          _ptr(scale_a), _ptr(scale_b), None if epi is None else ctypes.byref(epi),
                          _stream_ptr(stream))


def dg_gemv(x: dg_view, W: dg_view, y: dg_view, alpha: float, beta: float, stream=None) -> int:
    return lib.dg_gemv(ctypes.byref(x), ctypes.byref(W), ctypes.byref(y), float(alpha), float(beta),
                       _stream_ptr(stream))


def dg_gemv_w4(x: dg_view, W: dg_w4, y: dg_view, alpha: float, beta: float, epi=None, stream=None) -> int:
    """y = act(alpha * x W + beta * y + bias) for at most 8 rows and 4-bit weights; returns the status."""
    return lib.dg_gemv_w4(ctypes.byref(x), ctypes.byref(W), ctypes.byref(y), float(alpha), float(beta),
                          None if epi is None else ctypes.byref(epi), _stream_ptr(stream))


def dg_linear_ce(X: dg_view, W: dg_view, target, ignore_index: int, alpha: float, loss, lse, workspace,
                 workspace_bytes: int, stream=None) -> int:
    """loss and lse of the logits alpha * X W, which are not kept; returns the status."""
    return lib.dg_linear_ce(ctypes.byref(X), ctypes.byref(W), _ptr(target), int(ignore_index), float(alpha),
                            _ptr(loss), _ptr(lse), _ptr(workspace), int(workspace_bytes), _stream_ptr(stream))


def dg_linear_ce_grad(X: dg_view, W: dg_view, target, ignore_index: int, alpha: float, lse, dloss, dloss_stride: int,
                      dX, dW, workspace, workspace_bytes: int, stream=None) -> int:
    """dX and dW (dg_view or None) of sum_t dloss[t] * loss[t]; returns the status."""
    return lib.dg_linear_ce_grad(ctypes.byref(X), ctypes.byref(W), _ptr(target), int(ignore_index), float(alpha),
                                 _ptr(lse), _ptr(dloss), int(dloss_stride), None if dX is None else ctypes.byref(dX),
                                 None if dW is None else ctypes.byref(dW), _ptr(workspace), int(workspace_bytes),
                                 _stream_ptr(stream))


def dg_linear_ce_workspace(X: dg_view, W: dg_view):
    """(least, best): bytes of workspace dg_linear_ce needs and is fastest with."""
    least, best = ctypes.c_int64(), ctypes.c_int64()
    st = lib.dg_linear_ce_workspace(ctypes.byref(X), ctypes.byref(W), ctypes.byref(least), ctypes.byref(best))
    if st != DG_OK:
        raise DgError(st, "dg_linear_ce_workspace")
    return least.value, best.value


def dg_linear_ce_grad_workspace(X: dg_view, W: dg_view, dX=None, dW=None):
    """(least, best): bytes of workspace dg_linear_ce_grad needs and is fastest with."""
    least, best = ctypes.c_int64(), ctypes.c_int64()
    st = lib.dg_linear_ce_grad_workspace(ctypes.byref(X), ctypes.byref(W), None if dX is None else ctypes.byref(dX),
                                         None if dW is None else ctypes.byref(dW), ctypes.byref(least),
                                         ctypes.byref(best))
    if st != DG_OK:
        raise DgError(st, "dg_linear_ce_grad_workspace")
    return least.value, best.value


def dg_gemm_grouped(A: dg_view, B: dg_view, C: dg_view, offsets, groups: int, alpha: float, beta: float,
                    scale_a=None, scale_b=None, epi=None, stream=None) -> int:
    """C[r] = act(alpha * sa[r] * sb[g] * A[r] B[g] + beta * C[r] + bias[g]) for the rows r of each group g; returns
    the status."""
    return lib.dg_gemm_grouped(ctypes.byref(A), ctypes.byref(B), ctypes.byref(C), _ptr(offsets), int(groups),
                               float(alpha), float(beta), _ptr(scale_a), _ptr(scale_b),
                               None if epi is None else ctypes.byref(epi), _stream_ptr(stream))


def dg_gemm_grouped_dw(X: dg_view, dY: dg_view, dW: dg_view, offsets, groups: int, alpha: float, beta: float,
                       stream=None) -> int:
    """dW[g] = alpha * X^T dY over the rows of group g + beta * dW[g]; returns the status."""
    return lib.dg_gemm_grouped_dw(ctypes.byref(X), ctypes.byref(dY), ctypes.byref(dW), _ptr(offsets), int(groups),
                                  float(alpha), float(beta), _stream_ptr(stream))


def dg_mx4_scale_bytes(rows: int, K: int, block: int) -> int:
    """Bytes of the scales of a rows x K matrix of 4-bit floats (-1 for sizes that have none)."""
    return lib.dg_mx4_scale_bytes(int(rows), int(K), int(block))


def dg_quantize_mx4(x: dg_view, q: dg_mx4, stream=None) -> int:
    """Codes and scales of x; returns the status."""
    return lib.dg_quantize_mx4(ctypes.byref(x), ctypes.byref(q), _stream_ptr(stream))


def dg_dequantize_mx4(q: dg_mx4, y: dg_view, stream=None) -> int:
    """y = the values of q; returns the status."""
    return lib.dg_dequantize_mx4(ctypes.byref(q), ctypes.byref(y), _stream_ptr(stream))


def dg_gemm_mx4(A: dg_mx4, B: dg_mx4, C: dg_view, alpha: float, beta: float, epi=None, stream=None) -> int:
    """C = act(alpha * A B^T + beta * C + bias) of 4-bit floats; returns the status."""
    return lib.dg_gemm_mx4(ctypes.byref(A), ctypes.byref(B), ctypes.byref(C), float(alpha), float(beta),
                           None if epi is None else ctypes.byref(epi), _stream_ptr(stream))


def dg_sync_status(stream=None) -> int:
    return lib.dg_sync_status(_stream_ptr(stream))


def dg_analyse_view(v: dg_view) -> dg_view_info:
    out = dg_view_info()
    st = lib.dg_analyse_view(ctypes.byref(v), ctypes.byref(out))
    if st != DG_OK:
        raise DgError(st, "dg_analyse_view")
    return out


def dg_plan(A: dg_view, B: dg_view, C: dg_view, alpha=1.0, beta=0.0, has_scales=False,
            num_sms: int = 0) -> dg_plan_info:
    out = dg_plan_info()
    st = lib.dg_plan(ctypes.byref(A), ctypes.byref(B), ctypes.byref(C), float(alpha), float(beta),
                     int(bool(has_scales)), int(num_sms), ctypes.byref(out))
    if st != DG_OK:
        raise DgError(st, "dg_plan")
    return out


def dg_autotune(A: dg_view, B: dg_view, C: dg_view, alpha: float, beta: float, scale_a=None, scale_b=None,
                epi=None, stream=None, reps: int = 5):
    """Time the kernel variants for this call, keep the fastest for its shape
    key, and run the call: returns (status, dg_tune_result)."""
    out = dg_tune_result()
    st = lib.dg_autotune(ctypes.byref(A), ctypes.byref(B), ctypes.byref(C), float(alpha), float(beta),
                         _ptr(scale_a), _ptr(scale_b), None if epi is None else ctypes.byref(epi),
                         _stream_ptr(stream), int(reps), ctypes.byref(out))
    return st, out


def dg_tune_clear() -> None:
    lib.dg_tune_clear()


def dg_launch_count() -> int:
    return int(lib.dg_launch_count())


def dg_set_option(option: int, value: int) -> None:
    st = lib.dg_set_option(int(option), int(value))
    if st != DG_OK:
        raise DgError(st, "dg_set_option")


def dg_version() -> int:
    return int(lib.dg_version())


# ----------------------------------------------------------- conveniences

def _extents(x, row_dims: int):
    """Rows and columns of a torch tensor or dg_view."""
    shape = x.shape[:x.ndim]
    if isinstance(x, dg_view):
        row_dims = x.row_dims
    return math.prod(shape[:row_dims]), math.prod(shape[row_dims:])


def _floats(t, name: str, n: int):
    """A tensor that a kernel reads n floats of (an address is the caller's word for it)."""
    if t is None or isinstance(t, int):
        return
    if t.dtype != _torch.float32 or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous torch.float32 tensor of {n} elements")


def gemm(A, B, C, alpha: float = 1.0, beta: float = 0.0, scale_a=None, scale_b=None,
         stream=None, a_row_dims: int = 1, b_row_dims: int = 1, c_row_dims: int = 1,
         bias=None, act="none"):
    """dg_gemm (dg_gemm_ex when a bias or activation is given) on torch tensors
    or dg_view objects; raises DgError on a bad status.  scale_a, scale_b and
    bias are float32 of M, N and N elements at least."""
    if scale_a is not None or scale_b is not None or bias is not None:
        m, n = _extents(C, c_row_dims)
        _floats(scale_a, "scale_a", m)
        _floats(scale_b, "scale_b", n)
        _floats(bias, "bias", n)
    if bias is None and act in ("none", DG_ACT_NONE):
        st = dg_gemm(_as_view(A, a_row_dims), _as_view(B, b_row_dims), _as_view(C, c_row_dims),
                     alpha, beta, scale_a, scale_b, stream)
    else:
        st = dg_gemm_ex(_as_view(A, a_row_dims), _as_view(B, b_row_dims), _as_view(C, c_row_dims),
                        alpha, beta, scale_a, scale_b, epilogue(bias, act), stream)
    if st != DG_OK:
        raise DgError(st, "dg_gemm")
    return C


def gemv(x, W, y, alpha: float = 1.0, beta: float = 0.0, stream=None):
    st = dg_gemv(_as_view(x, 1), _as_view(W, 1), _as_view(y, 1), alpha, beta, stream)
    if st != DG_OK:
        raise DgError(st, "dg_gemv")
    return y


def w4(codes, scales, zeros=None, group: int = 128, K: int | None = None) -> dg_w4:
    """A dg_w4 of torch tensors in place: codes uint8 [N, ceil(K / 2)], two codes
    per byte along k (even k in the low four bits), scales [N, ceil(K / group)],
    zeros uint8 of the same shape or None (every zero point is 8).  K defaults
    to two per byte.  The last dim of each tensor must be contiguous."""
    import torch

    n, nbytes = codes.shape
    K = 2 * nbytes if K is None else int(K)
    groups = -(-K // group) if group > 0 else -1
    cs, ss = codes.stride(), scales.stride()
    zs = (0, 1) if zeros is None else zeros.stride()
    if codes.dtype != torch.uint8 or (zeros is not None and zeros.dtype != torch.uint8):
        raise TypeError("codes and zeros must be uint8")
    if nbytes != (K + 1) // 2:
        raise ValueError(f"codes must have ceil(K / 2) = {(K + 1) // 2} bytes a row, not {nbytes}")
    if scales.shape != (n, groups) or (zeros is not None and zeros.shape != (n, groups)):
        raise ValueError(f"scales and zeros must be [{n}, {groups}]")
    if (cs[1] != 1 and nbytes > 1) or ((ss[1] != 1 or zs[1] != 1) and groups > 1):
        raise ValueError("codes, scales and zeros must be contiguous along their last dim")
    code = _torch_dtype_code(scales)
    return dg_w4.from_buffer_copy(_W4.pack(codes.data_ptr(), scales.data_ptr(),
                                           0 if zeros is None else zeros.data_ptr(), K, n, cs[0],
                                           ss[0] * ELEM_SIZE[code], zs[0], int(group), code, 0, 0))


def gemv_w4(x, codes, scales, y, zeros=None, group: int = 128, alpha: float = 1.0, beta: float = 0.0,
            stream=None, bias=None, act="none"):
    """dg_gemv_w4 on torch tensors: y = act(alpha * x W + beta * y + bias), W [K x N]
    given by its codes, scales and zeros (see w4); x is [..., K] and y [..., N] with
    at most 8 rows, or [K] and [N].  Raises DgError on a bad status."""
    xv = view(x, x.dim() - 1)
    yv = view(y, y.dim() - 1)
    W = w4(codes, scales, zeros, group, x.shape[-1])
    _floats(bias, "bias", codes.shape[0])
    epi = None if bias is None and act in ("none", DG_ACT_NONE) else ctypes.byref(epilogue(bias, act))
    st = lib.dg_gemv_w4(ctypes.byref(xv), ctypes.byref(W), ctypes.byref(yv), alpha, beta, epi, _stream_ptr(stream))
    if st != DG_OK:
        raise DgError(st, "dg_gemv_w4")
    return y


class _Torch:
    """torch, imported on first use: the binding itself does not need it."""

    def __getattr__(self, name):
        import torch

        value = getattr(torch, name)
        setattr(self, name, value)
        return value


_torch = _Torch()


def _vector(t, name, dtype, n):
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements")
    return t


def _workspace(nbytes: int, stream):
    """Device bytes of torch's pool, allocated on the stream that uses them."""
    if stream is None:
        return _torch.empty(nbytes, dtype=_torch.uint8, device="cuda")
    if isinstance(stream, int):
        stream = _torch.cuda.ExternalStream(stream)
    with _torch.cuda.stream(stream):
        return _torch.empty(nbytes, dtype=_torch.uint8, device="cuda")


def linear_ce(x, w, target, loss, lse, alpha: float = 1.0, ignore_index: int = -100, stream=None, workspace=None,
              x_row_dims: int | None = None):
    """dg_linear_ce on torch tensors: the cross entropy of the logits alpha * x w
    against `target`, without keeping the logits.  x is [..., D] (its first
    x_row_dims dims, by default all but the last, are the rows and the others
    the features), w [D, V] (a [V, D] weight is passed as weight.t()), target
    int64, loss and lse float32, one per row.  `workspace` is a uint8 tensor (at
    least dg_linear_ce_workspace's bytes); None takes one from torch's pool.
    Raises DgError on a bad status; returns (loss, lse)."""
    rd = x.dim() - 1 if x_row_dims is None else x_row_dims
    xv, wv = view(x, rd), view(w)
    rows = x.shape[:rd].numel()
    _vector(target, "target", _torch.int64, rows)
    _vector(loss, "loss", _torch.float32, rows)
    _vector(lse, "lse", _torch.float32, rows)
    xr, wr = ctypes.byref(xv), ctypes.byref(wv)
    if workspace is None:
        least, best = ctypes.c_int64(), ctypes.c_int64()
        st = lib.dg_linear_ce_workspace(xr, wr, ctypes.byref(least), ctypes.byref(best))
        if st != DG_OK:
            raise DgError(st, "dg_linear_ce_workspace")
        workspace = _workspace(best.value, stream)
    st = lib.dg_linear_ce(xr, wr, target.data_ptr(), ignore_index, alpha, loss.data_ptr(), lse.data_ptr(),
                          workspace.data_ptr(), workspace.numel(), _stream_ptr(stream))
    if st != DG_OK:
        raise DgError(st, "dg_linear_ce")
    return loss, lse


def linear_ce_grad(x, w, target, lse, dloss, dx=None, dw=None, alpha: float = 1.0, ignore_index: int = -100,
                   stream=None, workspace=None, x_row_dims: int | None = None):
    """dg_linear_ce_grad on torch tensors: the gradients of sum(dloss * loss) into
    dx (like x) and dw (like w), either of which may be None.  dloss is float32,
    one per row, or one value for all rows (one element, or expanded from one);
    lse is what linear_ce wrote.  Raises DgError on a bad status; returns
    (dx, dw)."""
    rd = x.dim() - 1 if x_row_dims is None else x_row_dims
    xv, wv = view(x, rd), view(w)
    dxv = None if dx is None else view(dx, rd)
    dwv = None if dw is None else view(dw)
    rows = x.shape[:rd].numel()
    _vector(target, "target", _torch.int64, rows)
    _vector(lse, "lse", _torch.float32, rows)
    shared = dloss.numel() == 1 or not any(dloss.stride())  # one value, or expanded from one
    if not shared:
        _vector(dloss, "dloss", _torch.float32, rows)
    elif dloss.dtype != _torch.float32 or dloss.numel() not in (1, rows):
        raise ValueError(f"dloss must be a float32 tensor of 1 or {rows} elements")
    xr, wr = ctypes.byref(xv), ctypes.byref(wv)
    dxr, dwr = None if dx is None else ctypes.byref(dxv), None if dw is None else ctypes.byref(dwv)
    if workspace is None:
        least, best = ctypes.c_int64(), ctypes.c_int64()
        st = lib.dg_linear_ce_grad_workspace(xr, wr, dxr, dwr, ctypes.byref(least), ctypes.byref(best))
        if st != DG_OK:
            raise DgError(st, "dg_linear_ce_grad_workspace")
        workspace = _workspace(best.value, stream)
    st = lib.dg_linear_ce_grad(xr, wr, target.data_ptr(), ignore_index, alpha, lse.data_ptr(), dloss.data_ptr(),
                               0 if shared else 4, dxr, dwr, workspace.data_ptr(), workspace.numel(),
                               _stream_ptr(stream))
    if st != DG_OK:
        raise DgError(st, "dg_linear_ce_grad")
    return dx, dw


def _groups(offsets, stack) -> int:
    """The number of groups, from int64 offsets [groups + 1] and a [groups, K, N] tensor."""
    size, shape = offsets.shape, stack.shape
    if len(size) != 1 or size[0] < 1 or offsets.dtype != _torch.int64 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int64 tensor of groups + 1 elements")
    if len(shape) != 3 or shape[0] != size[0] - 1:
        raise ValueError(f"expected [{size[0] - 1}, K, N], got {tuple(shape)}")
    return shape[0]


def gemm_grouped(a, b, c, offsets, scale_a=None, scale_b=None, alpha: float = 1.0, beta: float = 0.0, bias=None,
                 act="none", stream=None):
    """dg_gemm_grouped on torch tensors: c[r] = act(alpha * scale_a[r] * scale_b[g] * (a[r] b[g]) + beta * c[r] +
    bias[g]) for the rows r of each group g, offsets[g] <= r < offsets[g + 1].  a is [..., K] (R rows in all), b
    [groups, K, N] (a [groups, N, K] weight is passed as weight.transpose(1, 2)), c [..., N], offsets int64
    [groups + 1] on the device; scale_a float32 [R], scale_b and bias float32 [groups, N].  Raises DgError on a bad
    status; returns c."""
    groups = _groups(offsets, b)
    if scale_a is not None:
        _vector(scale_a, "scale_a", _torch.float32, a.shape[:-1].numel())
    for name, t in (("scale_b", scale_b), ("bias", bias)):
        if t is not None:
            _vector(t, name, _torch.float32, groups * b.shape[2])
    epi = None if bias is None and act in ("none", DG_ACT_NONE) else ctypes.byref(epilogue(bias, act))
    st = lib.dg_gemm_grouped(_packed_view(a, a.dim() - 1), _packed_view(b, 2), _packed_view(c, c.dim() - 1),
                             offsets.data_ptr(), groups, alpha, beta, _ptr(scale_a), _ptr(scale_b), epi,
                             _stream_ptr(stream))
    if st != DG_OK:
        raise DgError(st, "dg_gemm_grouped")
    return c


def gemm_grouped_dw(x, dy, dw, offsets, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """dg_gemm_grouped_dw on torch tensors: dw[g] = alpha * x^T dy over the rows of group g + beta * dw[g].  x is
    [..., K], dy [..., N], dw [groups, K, N] (that of a [groups, N, K] weight is passed as dweight.transpose(1, 2)).
    Raises DgError on a bad status; returns dw."""
    groups = _groups(offsets, dw)
    st = lib.dg_gemm_grouped_dw(_packed_view(x, x.dim() - 1), _packed_view(dy, dy.dim() - 1), _packed_view(dw, 2),
                                offsets.data_ptr(), groups, alpha, beta, _stream_ptr(stream))
    if st != DG_OK:
        raise DgError(st, "dg_gemm_grouped_dw")
    return dw


def empty_mx4(rows: int, K: int, block: int = 32, device="cuda"):
    """(codes, scales): uninitialised tensors for a rows x K matrix of 4-bit floats, its rows of codes at multiples of
    16 bytes, as gemm_mx4 wants them.  (K odd: quantize_mx4 zeroes the last byte's unused half.)"""
    codes = _torch.empty(rows, (K + 31) // 32 * 16, dtype=_torch.uint8, device=device)[:, :(K + 1) // 2]
    return codes, _torch.empty(max(0, dg_mx4_scale_bytes(rows, K, block)), dtype=_torch.uint8, device=device)


def mx4(codes, scales, K: int | None = None, block: int = 32, scale=None) -> dg_mx4:
    """A dg_mx4 of torch tensors in place: codes uint8 [rows, ceil(K / 2)], two E2M1 codes per byte along k (even k in
    the low four bits), scales uint8 in tiles (dg_mx4_scale_bytes of them), scale a float32 of one element on the
    device or None.  K defaults to two per byte."""
    return dg_mx4.from_buffer_copy(_packed_mx4(codes, scales, K, block, scale))


def _packed_mx4(codes, scales, K, block, scale) -> bytes:
    rows, nbytes = codes.shape
    K = 2 * nbytes if K is None else int(K)
    stride = codes.stride()
    if codes.dtype != _torch.uint8 or scales.dtype != _torch.uint8:
        raise TypeError("codes and scales must be uint8")
    if nbytes != (K + 1) // 2 or (nbytes > 1 and stride[1] != 1):
        raise ValueError(f"codes must have ceil(K / 2) = {(K + 1) // 2} contiguous bytes a row")
    if block not in (16, 32):
        raise ValueError("block must be 16 or 32")
    need = -(-rows // 128) * -(-K // (4 * block)) * 512  # dg_mx4_scale_bytes
    if scales.numel() != need or not scales.is_contiguous():
        raise ValueError(f"scales must be {need} contiguous bytes (block {block})")
    if scale is not None:
        _vector(scale, "scale", _torch.float32, 1)
    return _MX4.pack(codes.data_ptr(), scales.data_ptr(), 0 if scale is None else scale.data_ptr(), rows, K, stride[0],
                     block, 0)


def quantize_mx4(x, codes, scales, block: int = 32, scale=None, stream=None):
    """dg_quantize_mx4 on torch tensors: the codes and block scales (see mx4) of x [..., K] / scale, written in
    place.  Raises DgError on a bad status; returns (codes, scales)."""
    st = lib.dg_quantize_mx4(_packed_view(x, x.dim() - 1), _packed_mx4(codes, scales, x.shape[-1], block, scale),
                             _stream_ptr(stream))
    if st != DG_OK:
        raise DgError(st, "dg_quantize_mx4")
    return codes, scales


def dequantize_mx4(codes, scales, y, block: int = 32, scale=None, stream=None):
    """dg_dequantize_mx4 on torch tensors: y [..., K] = the values of codes and scales (see mx4).  Raises DgError on
    a bad status; returns y."""
    st = lib.dg_dequantize_mx4(_packed_mx4(codes, scales, y.shape[-1], block, scale), _packed_view(y, y.dim() - 1),
                               _stream_ptr(stream))
    if st != DG_OK:
        raise DgError(st, "dg_dequantize_mx4")
    return y


def gemm_mx4(a: dg_mx4, b: dg_mx4, c, alpha: float = 1.0, beta: float = 0.0, bias=None, act="none", stream=None):
    """dg_gemm_mx4: c [M, N] = act(alpha * a b^T + beta * c + bias) of a [M, K] and b [N, K] in 4-bit floats (see
    mx4), c a torch tensor or dg_view, bias float32 [N].  Raises DgError on a bad status; returns c."""
    if bias is not None and not isinstance(bias, int):
        _vector(bias, "bias", _torch.float32, b.rows)
    cv = ctypes.byref(c) if isinstance(c, dg_view) else _packed_view(c, 1)
    epi = None if bias is None and act in ("none", DG_ACT_NONE) else ctypes.byref(epilogue(bias, act))
    st = lib.dg_gemm_mx4(ctypes.byref(a), ctypes.byref(b), cv, alpha, beta, epi, _stream_ptr(stream))
    if st != DG_OK:
        raise DgError(st, "dg_gemm_mx4")
    return c
