"""Python binding of the MXFP8 C-ABI library (include/mxfp8.h).

Argument marshalling only: every step of quantisation and GEMM runs in the
library's sm_103a kernels. PyTorch supplies device memory and streams. If the
shared library has not been built, importing the binding's functions raises;
there is no fallback path.

The raw entry points keep the C names (``mx_quantize``, ``mx_gemm``,
``mx_grouped_gemm``, ``mx_scale_bytes``, ``mx_grouped_padded_rows``,
``mx_status_string``, ``mx_last_error``, ``mx_abi_version``) and take integer
device pointers. ``quantize`` / ``gemm`` / ``grouped_gemm`` wrap them for
torch tensors, allocating outputs with torch. A wrapper launches on the current
stream, or on the ``stream`` it is given; its outputs and scratch belong to that
stream, as if it had been called under ``torch.cuda.stream(stream)``.
"""

from __future__ import annotations

import ctypes
import itertools
import os
import struct
from dataclasses import dataclass
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmxfp8_gb300.so")

MX_ROWWISE, MX_COLWISE, MX_BOTH = 1, 2, 3
MX_FPROP, MX_DGRAD, MX_WGRAD = 0, 1, 2
MX_MAX_MULTI = 8
MX_MAX_GEMM_MULTI = 4
MX_MAX_GROUPS = 512
MX_BF16, MX_F32 = 0, 1
MX_ADAMW_STATE_BLOCK = 256
MX_ADD_NORM_MAX_COLS = 16384
MX_ACT_NONE, MX_ACT_RELU, MX_ACT_GELU, MX_ACT_SILU = 0, 1, 2, 3
ACTIVATIONS = {"none": MX_ACT_NONE, "relu": MX_ACT_RELU, "gelu": MX_ACT_GELU, "silu": MX_ACT_SILU}
STATUS_NAMES = {0: "MX_OK", 1: "MX_ERR_INVALID_ARG", 2: "MX_ERR_UNSUPPORTED_SHAPE", 3: "MX_ERR_ALIGNMENT",
                4: "MX_ERR_CUDA", 5: "MX_ERR_DEVICE_CHECK", 6: "MX_ERR_TIMEOUT", 7: "MX_ERR_NO_DEVICE"}

# Symbols the header declares (the CPU tests check the library exports them).
EXPORTED = ("mx_scale_bytes", "mx_grouped_padded_rows", "mx_quantize", "mx_quantize_batched", "mx_quantize_f32",
            "mx_quantize_multi",
            "mx_gemm", "mx_grouped_gemm", "mx_grouped_gemm_swiglu", "mx_quantize_fp8_blockwise",
            "mx_gemm_fp8_blockwise", "mx_status_string", "mx_last_error", "mx_abi_version",
            "mx_selftest_wait_timeout", "mx_gemm_workspace_bytes", "mx_gemm_with_workspace", "mx_gemm_multi",
            "mx_gemm_static_workspace", "mx_current_amax", "mx_quantize_current", "mx_gemm_current",
            "mx_grouped_gemm_current", "mx_gemm_current_multi", "mx_grouped_gemm_swiglu_quantize", "mx_adamw_step",
            "mx_layer_norm", "mx_layer_norm_backward_workspace_bytes", "mx_layer_norm_backward",
            "mx_gemm_epilogue", "mx_epilogue_backward_workspace_bytes", "mx_epilogue_backward",
            "mx_router_workspace_bytes", "mx_router_forward", "mx_router_backward", "mx_selftest_norm_timeout",
            "mx_add_norm_quantize", "mx_add_norm_backward_workspace_bytes", "mx_add_norm_backward", "mx_gemm_gated",
            "mx_gated_quantize", "mx_gated_backward_quantize", "mx_selftest_block_timeout")
MX_STATIC_WORKSPACE_BYTES = 40 * 1024 * 1024


class MXError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}" + (f" ({detail})" if detail else ""))


class MXOperandC(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("k", ctypes.c_int64), ("ld", ctypes.c_int64), ("orient", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class MXGemmProblemC(ctypes.Structure):
    _fields_ = [("a", MXOperandC), ("b", MXOperandC), ("c", ctypes.c_void_p), ("ldc", ctypes.c_int64),
                ("mode", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MXQuantTensorC(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ldx", ctypes.c_int64),
                ("row_data", ctypes.c_void_p), ("row_scale", ctypes.c_void_p), ("col_data", ctypes.c_void_p),
                ("col_scale", ctypes.c_void_p)]


class MXEpilogueC(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("preact", ctypes.c_void_p),
                ("ld_residual", ctypes.c_int64), ("ld_preact", ctypes.c_int64), ("bias_dtype", ctypes.c_int32),
                ("act", ctypes.c_int32)]


class MXAdamWTensorC(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("numel", ctypes.c_int64), ("weight_decay", ctypes.c_double),
                ("grad_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MXAdamWHyperC(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("seed", ctypes.c_uint32),
                ("reserved", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load the shared library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m mxfp8_block_scaled_gb300.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.mx_scale_bytes.argtypes = [i64, i64]
    L.mx_scale_bytes.restype = ctypes.c_size_t
    L.mx_grouped_padded_rows.argtypes = [ctypes.POINTER(ctypes.c_int64), i32]
    L.mx_grouped_padded_rows.restype = i64
    L.mx_quantize.argtypes = [vp, i64, i64, i64, i32, vp, vp, vp, vp, vp, i32, i64, vp, vp]
    L.mx_quantize.restype = i32
    L.mx_quantize_batched.argtypes = [vp, i64, i64, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp]
    L.mx_quantize_batched.restype = i32
    L.mx_quantize_f32.argtypes = [vp, i64, i64, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp]
    L.mx_quantize_f32.restype = i32
    L.mx_quantize_multi.argtypes = [ctypes.POINTER(MXQuantTensorC), i32, i32, vp, vp]
    L.mx_quantize_multi.restype = i32
    L.mx_gemm.argtypes = [i32, ctypes.POINTER(MXOperandC), ctypes.POINTER(MXOperandC), vp, i64, vp, vp]
    L.mx_gemm.restype = i32
    L.mx_gemm_workspace_bytes.argtypes = [i32, ctypes.POINTER(MXOperandC), ctypes.POINTER(MXOperandC),
                                          ctypes.POINTER(ctypes.c_size_t)]
    L.mx_gemm_workspace_bytes.restype = i32
    L.mx_gemm_with_workspace.argtypes = [i32, ctypes.POINTER(MXOperandC), ctypes.POINTER(MXOperandC), vp, i64, vp,
                                         ctypes.c_size_t, vp, vp]
    L.mx_gemm_with_workspace.restype = i32
    L.mx_gemm_static_workspace.argtypes = [i32, ctypes.POINTER(MXOperandC), ctypes.POINTER(MXOperandC), vp, i64,
                                           vp, vp]
    L.mx_gemm_static_workspace.restype = i32
    L.mx_current_amax.argtypes = [vp, i64, i64, i64, i64, i64, vp, vp, vp]
    L.mx_current_amax.restype = i32
    L.mx_quantize_current.argtypes = [vp, i64, i64, i64, i64, i64, i32, vp, ctypes.c_float, vp, vp, vp, vp, i32, i64,
                                      vp, vp]
    L.mx_quantize_current.restype = i32
    L.mx_gemm_current.argtypes = [i32, ctypes.POINTER(MXOperandC), ctypes.POINTER(MXOperandC), vp, i64, vp, vp]
    L.mx_gemm_current.restype = i32
    L.mx_grouped_gemm_current.argtypes = [i32, ctypes.POINTER(MXOperandC), ctypes.POINTER(MXOperandC), vp, i32, vp,
                                          i64, vp, vp]
    L.mx_grouped_gemm_current.restype = i32
    L.mx_gemm_multi.argtypes = [ctypes.POINTER(MXGemmProblemC), i32, vp, vp]
    L.mx_gemm_multi.restype = i32
    L.mx_gemm_current_multi.argtypes = [ctypes.POINTER(MXGemmProblemC), i32, vp, vp]
    L.mx_gemm_current_multi.restype = i32
    L.mx_grouped_gemm.argtypes = [i32, ctypes.POINTER(MXOperandC), ctypes.POINTER(MXOperandC), vp, i32, vp, i64,
                                  vp, vp]
    L.mx_grouped_gemm.restype = i32
    L.mx_grouped_gemm_swiglu.argtypes = [ctypes.POINTER(MXOperandC), ctypes.POINTER(MXOperandC), vp, i32, vp, i64,
                                         vp, vp]
    L.mx_grouped_gemm_swiglu.restype = i32
    L.mx_grouped_gemm_swiglu_quantize.argtypes = [ctypes.POINTER(MXOperandC), ctypes.POINTER(MXOperandC), vp, i32, vp,
                                                  vp, vp, vp, i64, vp, vp]
    L.mx_grouped_gemm_swiglu_quantize.restype = i32
    L.mx_quantize_fp8_blockwise.argtypes = [vp, i64, i64, i64, i32, vp, vp, vp, vp]
    L.mx_quantize_fp8_blockwise.restype = i32
    L.mx_gemm_fp8_blockwise.argtypes = [vp, vp, i64, vp, vp, i64, i64, vp, i64, vp, vp]
    L.mx_gemm_fp8_blockwise.restype = i32
    L.mx_adamw_step.argtypes = [vp, i32, i32, ctypes.POINTER(MXAdamWHyperC), vp, vp, vp]
    L.mx_adamw_step.restype = i32
    L.mx_layer_norm.argtypes = [vp, i64, vp, vp, i32, i64, i64, ctypes.c_float, i32, i32, vp, i64, vp, vp, vp, vp]
    L.mx_layer_norm.restype = i32
    L.mx_layer_norm_backward_workspace_bytes.argtypes = [i64, i64]
    L.mx_layer_norm_backward_workspace_bytes.restype = ctypes.c_size_t
    L.mx_layer_norm_backward.argtypes = [vp, i64, vp, i64, vp, i32, vp, vp, i64, i64, i32, i32, vp, i64, vp, vp, vp,
                                         ctypes.c_size_t, vp, vp]
    L.mx_layer_norm_backward.restype = i32
    L.mx_gemm_epilogue.argtypes = [i32, ctypes.POINTER(MXOperandC), ctypes.POINTER(MXOperandC),
                                   ctypes.POINTER(MXEpilogueC), vp, i64, vp, vp]
    L.mx_gemm_epilogue.restype = i32
    L.mx_epilogue_backward_workspace_bytes.argtypes = [i64, i64]
    L.mx_epilogue_backward_workspace_bytes.restype = ctypes.c_size_t
    L.mx_epilogue_backward.argtypes = [vp, i64, vp, i64, i64, i64, i32, vp, i64, vp, vp, ctypes.c_size_t, vp, vp]
    L.mx_epilogue_backward.restype = i32
    L.mx_router_workspace_bytes.argtypes = [i64, i64, i32]
    L.mx_router_workspace_bytes.restype = ctypes.c_size_t
    L.mx_router_forward.argtypes = [vp, i64, i32, vp, i64, i64, i32, i32, i32, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp,
                                    ctypes.c_size_t, vp, vp]
    L.mx_router_forward.restype = i32
    L.mx_router_backward.argtypes = [vp, i64, i32, vp, i64, i64, i32, i32, i32, vp, vp, vp, vp, vp, i64, vp, vp]
    L.mx_router_backward.restype = i32
    L.mx_add_norm_quantize.argtypes = [vp, i64, vp, i64, i32, vp, i32, i64, i64, ctypes.c_float, i32, vp, i64, vp, i64, vp,
                                       vp, vp, vp, vp, vp, vp]
    L.mx_add_norm_quantize.restype = i32
    L.mx_add_norm_backward_workspace_bytes.argtypes = [i64, i64]
    L.mx_add_norm_backward_workspace_bytes.restype = ctypes.c_size_t
    L.mx_add_norm_backward.argtypes = [vp, i64, vp, i64, vp, i64, i32, vp, i32, vp, i64, i64, i32, vp, i64, vp, vp, vp, vp,
                                       vp, vp, ctypes.c_size_t, vp, vp]
    L.mx_add_norm_backward.restype = i32
    L.mx_gemm_gated.argtypes = [ctypes.POINTER(MXOperandC), ctypes.POINTER(MXOperandC), ctypes.POINTER(MXOperandC), i32,
                                vp, i64, vp, i64, vp, vp]
    L.mx_gemm_gated.restype = i32
    L.mx_gated_quantize.argtypes = [vp, i64, i64, i64, i32, i32, vp, vp, vp, vp, vp, i32, i64, vp, vp]
    L.mx_gated_quantize.restype = i32
    L.mx_gated_backward_quantize.argtypes = [vp, i64, vp, i64, i64, i64, i32, i32, vp, vp, vp, vp, vp, i32, i64, vp, vp]
    L.mx_gated_backward_quantize.restype = i32
    L.mx_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp, vp]
    L.mx_selftest_wait_timeout.restype = i32
    L.mx_selftest_norm_timeout.argtypes = [ctypes.c_uint64, vp, vp, i64, i64, vp, vp, vp, vp, vp, ctypes.c_size_t, vp, vp]
    L.mx_selftest_norm_timeout.restype = i32
    L.mx_selftest_block_timeout.argtypes = [i32, ctypes.c_uint64]
    L.mx_selftest_block_timeout.restype = i32
    L.mx_status_string.argtypes = [i32]
    L.mx_status_string.restype = ctypes.c_char_p
    L.mx_last_error.argtypes = []
    L.mx_last_error.restype = ctypes.c_char_p
    L.mx_abi_version.argtypes = []
    L.mx_abi_version.restype = i32
    _lib = L
    return L


def _check(status: int, where: str) -> None:
    if status != 0:
        raise MXError(status, where, lib().mx_last_error().decode(errors="replace"))


# ---------------------------------------------------------------------------
# Raw entry points (same names as the C ABI; integer device pointers)
# ---------------------------------------------------------------------------

def mx_scale_bytes(rows: int, k: int) -> int:
    return int(lib().mx_scale_bytes(rows, k))


def mx_grouped_padded_rows(host_offsets) -> int:
    offs = [int(v) for v in host_offsets]
    arr = (ctypes.c_int64 * len(offs))(*offs)
    return int(lib().mx_grouped_padded_rows(arr, len(offs) - 1))


def mx_status_string(status: int) -> str:
    return lib().mx_status_string(status).decode()


def mx_last_error() -> str:
    return lib().mx_last_error().decode(errors="replace")


def mx_abi_version() -> int:
    return int(lib().mx_abi_version())


def mx_quantize(x, rows, cols, ldx, axis, row_data, row_scale, col_data, col_scale, group_offsets, n_groups,
                col_capacity, dev_status, stream) -> None:
    _check(lib().mx_quantize(x, rows, cols, ldx, axis, row_data, row_scale, col_data, col_scale, group_offsets,
                             n_groups, col_capacity, dev_status, stream), "mx_quantize")


def mx_quantize_batched(x, batch, rows, cols, ldx, x_batch_stride, axis, row_data, row_scale, col_data, col_scale,
                        dev_status, stream) -> None:
    _check(lib().mx_quantize_batched(x, batch, rows, cols, ldx, x_batch_stride, axis, row_data, row_scale, col_data,
                                     col_scale, dev_status, stream), "mx_quantize_batched")


def mx_quantize_f32(x, batch, rows, cols, ldx, x_batch_stride, axis, row_data, row_scale, col_data, col_scale,
                    dev_status, stream) -> None:
    _check(lib().mx_quantize_f32(x, batch, rows, cols, ldx, x_batch_stride, axis, row_data, row_scale, col_data,
                                 col_scale, dev_status, stream), "mx_quantize_f32")


def mx_quantize_multi(tensors, axis, dev_status, stream) -> None:
    """``tensors``: a sequence of MXQuantTensorC."""
    arr = (MXQuantTensorC * max(len(tensors), 1))(*tensors)
    _check(lib().mx_quantize_multi(arr, len(tensors), axis, dev_status, stream), "mx_quantize_multi")


def mx_quantize_fp8_blockwise(x, rows, cols, ldx, block, data, scale, dev_status, stream) -> None:
    _check(lib().mx_quantize_fp8_blockwise(x, rows, cols, ldx, block, data, scale, dev_status, stream),
           "mx_quantize_fp8_blockwise")


def mx_gemm_fp8_blockwise(a_data, a_scale, M, b_data, b_scale, N, K, c, ldc, dev_status, stream) -> None:
    _check(lib().mx_gemm_fp8_blockwise(a_data, a_scale, M, b_data, b_scale, N, K, c, ldc, dev_status, stream),
           "mx_gemm_fp8_blockwise")


def mx_selftest_wait_timeout(timeout_ns, dev_status, stream) -> None:
    _check(lib().mx_selftest_wait_timeout(timeout_ns, dev_status, stream), "mx_selftest_wait_timeout")


def mx_selftest_norm_timeout(timeout_ns, dy, x, rows, cols, out, rstd, dweight, dbias, workspace, workspace_bytes, dev_status,
                             stream) -> None:
    _check(lib().mx_selftest_norm_timeout(timeout_ns, dy, x, rows, cols, out, rstd, dweight, dbias, workspace,
                                          workspace_bytes, dev_status, stream), "mx_selftest_norm_timeout")


def mx_selftest_block_timeout(what, timeout_ns) -> None:
    _check(lib().mx_selftest_block_timeout(what, timeout_ns), "mx_selftest_block_timeout")


def _ref(op):
    return None if op is None else ctypes.byref(op)


def mx_gemm(mode, a: MXOperandC, b: MXOperandC, c, ldc, dev_status, stream) -> None:
    _check(lib().mx_gemm(mode, _ref(a), _ref(b), c, ldc, dev_status, stream), "mx_gemm")


def mx_gemm_workspace_bytes(mode, a: MXOperandC, b: MXOperandC) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().mx_gemm_workspace_bytes(mode, _ref(a), _ref(b), ctypes.byref(out)), "mx_gemm_workspace_bytes")
    return int(out.value)


def mx_gemm_with_workspace(mode, a: MXOperandC, b: MXOperandC, c, ldc, workspace, workspace_bytes, dev_status,
                           stream) -> None:
    _check(lib().mx_gemm_with_workspace(mode, _ref(a), _ref(b), c, ldc, workspace, workspace_bytes, dev_status,
                                        stream), "mx_gemm_with_workspace")


def mx_gemm_static_workspace(mode, a: MXOperandC, b: MXOperandC, c, ldc, dev_status, stream) -> None:
    _check(lib().mx_gemm_static_workspace(mode, _ref(a), _ref(b), c, ldc, dev_status, stream),
           "mx_gemm_static_workspace")


def mx_current_amax(x, batch, rows, cols, ldx, x_batch_stride, amax, dev_status, stream) -> None:
    _check(lib().mx_current_amax(x, batch, rows, cols, ldx, x_batch_stride, amax, dev_status, stream),
           "mx_current_amax")


def mx_quantize_current(x, batch, rows, cols, ldx, x_batch_stride, axis, amax, format_max, row_data, col_data, scale,
                        group_offsets, n_groups, col_capacity, dev_status, stream) -> None:
    _check(lib().mx_quantize_current(x, batch, rows, cols, ldx, x_batch_stride, axis, amax, format_max, row_data,
                                     col_data, scale, group_offsets, n_groups, col_capacity, dev_status, stream),
           "mx_quantize_current")


def mx_gemm_current(mode, a: MXOperandC, b: MXOperandC, c, ldc, dev_status, stream) -> None:
    _check(lib().mx_gemm_current(mode, _ref(a), _ref(b), c, ldc, dev_status, stream), "mx_gemm_current")


def mx_grouped_gemm_current(mode, a: MXOperandC, b: MXOperandC, group_offsets, n_groups, c, ldc, dev_status,
                            stream) -> None:
    _check(lib().mx_grouped_gemm_current(mode, _ref(a), _ref(b), group_offsets, n_groups, c, ldc, dev_status, stream),
           "mx_grouped_gemm_current")


def mx_gemm_multi(problems, dev_status, stream) -> None:
    """``problems``: a sequence of MXGemmProblemC."""
    arr = (MXGemmProblemC * max(len(problems), 1))(*problems)
    _check(lib().mx_gemm_multi(arr, len(problems), dev_status, stream), "mx_gemm_multi")


def mx_gemm_current_multi(problems, dev_status, stream) -> None:
    """``problems``: a sequence of MXGemmProblemC over current-scaled operands."""
    arr = (MXGemmProblemC * max(len(problems), 1))(*problems)
    _check(lib().mx_gemm_current_multi(arr, len(problems), dev_status, stream), "mx_gemm_current_multi")


def mx_grouped_gemm(mode, a: MXOperandC, b: MXOperandC, group_offsets, n_groups, c, ldc, dev_status,
                    stream) -> None:
    _check(lib().mx_grouped_gemm(mode, _ref(a), _ref(b), group_offsets, n_groups, c, ldc,
                                 dev_status, stream), "mx_grouped_gemm")


def mx_grouped_gemm_swiglu(a: MXOperandC, b: MXOperandC, group_offsets, n_groups, c, ldc, dev_status,
                           stream) -> None:
    _check(lib().mx_grouped_gemm_swiglu(_ref(a), _ref(b), group_offsets, n_groups, c, ldc, dev_status, stream),
           "mx_grouped_gemm_swiglu")


def mx_grouped_gemm_swiglu_quantize(a: MXOperandC, b: MXOperandC, group_offsets, n_groups, row_data, row_scale,
                                    col_data, col_scale, col_capacity, dev_status, stream) -> None:
    _check(lib().mx_grouped_gemm_swiglu_quantize(_ref(a), _ref(b), group_offsets, n_groups, row_data, row_scale,
                                                 col_data, col_scale, col_capacity, dev_status, stream),
           "mx_grouped_gemm_swiglu_quantize")


def mx_adamw_step(tensors, n, state_bits, hyper: MXAdamWHyperC, grad_scale, dev_status, stream) -> None:
    """``tensors``: an array of n MXAdamWTensorC, or the bytes of one."""
    _check(lib().mx_adamw_step(tensors, n, state_bits, _ref(hyper), grad_scale, dev_status, stream), "mx_adamw_step")


def mx_layer_norm(x, ldx, weight, bias, param_dtype, rows, cols, eps, center, dtype, y, ldy, mean, rstd, dev_status,
                  stream) -> None:
    _check(lib().mx_layer_norm(x, ldx, weight, bias, param_dtype, rows, cols, eps, center, dtype, y, ldy, mean, rstd,
                               dev_status, stream), "mx_layer_norm")


def mx_layer_norm_backward_workspace_bytes(rows, cols) -> int:
    return int(lib().mx_layer_norm_backward_workspace_bytes(rows, cols))


def mx_layer_norm_backward(dy, lddy, x, ldx, weight, param_dtype, mean, rstd, rows, cols, center, dtype, dx, lddx,
                           dweight, dbias, workspace, workspace_bytes, dev_status, stream) -> None:
    _check(lib().mx_layer_norm_backward(dy, lddy, x, ldx, weight, param_dtype, mean, rstd, rows, cols, center, dtype,
                                        dx, lddx, dweight, dbias, workspace, workspace_bytes, dev_status, stream),
           "mx_layer_norm_backward")


def mx_gemm_epilogue(mode, a: MXOperandC, b: MXOperandC, epilogue: MXEpilogueC, c, ldc, dev_status, stream) -> None:
    _check(lib().mx_gemm_epilogue(mode, _ref(a), _ref(b), _ref(epilogue), c, ldc, dev_status, stream),
           "mx_gemm_epilogue")


def mx_epilogue_backward_workspace_bytes(rows, cols) -> int:
    return int(lib().mx_epilogue_backward_workspace_bytes(rows, cols))


def mx_epilogue_backward(dy, lddy, preact, ld_preact, rows, cols, act, dz, lddz, dbias, workspace, workspace_bytes,
                         dev_status, stream) -> None:
    _check(lib().mx_epilogue_backward(dy, lddy, preact, ld_preact, rows, cols, act, dz, lddz, dbias, workspace,
                                      workspace_bytes, dev_status, stream), "mx_epilogue_backward")


def mx_router_workspace_bytes(tokens, tokens_per_seq, n_experts) -> int:
    return int(lib().mx_router_workspace_bytes(tokens, tokens_per_seq, n_experts))


def mx_router_forward(logits, ld, dtype, token_mask, tokens, tokens_per_seq, n_experts, top_k, normalize, coef, indices,
                      weights, counts, group_offsets, load, loss, workspace, workspace_bytes, dev_status,
                      stream) -> None:
    _check(lib().mx_router_forward(logits, ld, dtype, token_mask, tokens, tokens_per_seq, n_experts, top_k, normalize,
                                   coef, indices, weights, counts, group_offsets, load, loss, workspace,
                                   workspace_bytes, dev_status, stream), "mx_router_forward")


def mx_router_backward(logits, ld, dtype, token_mask, tokens, tokens_per_seq, n_experts, top_k, normalize, indices, load,
                       dweights, dloss, dlogits, lddx, dev_status, stream) -> None:
    _check(lib().mx_router_backward(logits, ld, dtype, token_mask, tokens, tokens_per_seq, n_experts, top_k, normalize,
                                    indices, load, dweights, dloss, dlogits, lddx, dev_status, stream),
           "mx_router_backward")


def mx_add_norm_quantize(x, ldx, residual, ld_residual, stream_dtype, weight, param_dtype, rows, cols, eps, axis, sum,
                         ld_sum, y, ldy, rstd, row_data, row_scale, col_data, col_scale, dev_status, stream) -> None:
    _check(lib().mx_add_norm_quantize(x, ldx, residual, ld_residual, stream_dtype, weight, param_dtype, rows, cols, eps,
                                      axis, sum, ld_sum, y, ldy, rstd, row_data, row_scale, col_data, col_scale,
                                      dev_status, stream), "mx_add_norm_quantize")


def mx_add_norm_backward_workspace_bytes(rows, cols) -> int:
    return int(lib().mx_add_norm_backward_workspace_bytes(rows, cols))


def mx_add_norm_backward(dy, lddy, sum, ld_sum, dsum, ld_dsum, stream_dtype, weight, param_dtype, rstd, rows, cols, axis,
                         dx, lddx, dweight, row_data, row_scale, col_data, col_scale, workspace, workspace_bytes,
                         dev_status, stream) -> None:
    _check(lib().mx_add_norm_backward(dy, lddy, sum, ld_sum, dsum, ld_dsum, stream_dtype, weight, param_dtype, rstd, rows,
                                      cols, axis, dx, lddx, dweight, row_data, row_scale, col_data, col_scale, workspace,
                                      workspace_bytes, dev_status, stream), "mx_add_norm_backward")


def mx_gemm_gated(a: MXOperandC, gate: MXOperandC, up: MXOperandC, act, c, ldc, preact, ld_preact, dev_status,
                  stream) -> None:
    _check(lib().mx_gemm_gated(_ref(a), _ref(gate), _ref(up), act, c, ldc, preact, ld_preact, dev_status, stream),
           "mx_gemm_gated")


def mx_gated_quantize(gate_up, ld, rows, f, act, axis, row_data, row_scale, col_data, col_scale, group_offsets, n_groups,
                      col_capacity, dev_status, stream) -> None:
    _check(lib().mx_gated_quantize(gate_up, ld, rows, f, act, axis, row_data, row_scale, col_data, col_scale,
                                   group_offsets, n_groups, col_capacity, dev_status, stream), "mx_gated_quantize")


def mx_gated_backward_quantize(dh, lddh, gate_up, ld, rows, f, act, axis, row_data, row_scale, col_data, col_scale,
                               group_offsets, n_groups, col_capacity, dev_status, stream) -> None:
    _check(lib().mx_gated_backward_quantize(dh, lddh, gate_up, ld, rows, f, act, axis, row_data, row_scale, col_data,
                                            col_scale, group_offsets, n_groups, col_capacity, dev_status, stream),
           "mx_gated_backward_quantize")


# ---------------------------------------------------------------------------
# torch-tensor wrappers
# ---------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _given(t) -> Optional[int]:
    """The address of a tensor that a caller may give; a CPU tensor's must not reach a kernel."""
    if t is None:
        return None
    assert t.is_cuda, "status and group_offsets: CUDA tensors"
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream.cuda_stream
    # The current stream of the current device, without building a Stream object
    # (3 us of a call's 10 on the host).
    c = _torch()._C
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


def _output(t):
    """A given output's address, likewise."""
    assert t.is_cuda, "out: a CUDA tensor"
    return t.data_ptr()


def _under(stream, wrapper, arguments):
    """Calls a wrapper again under the stream it was given, so that what it
    allocates (outputs, and scratch that is dropped on return while the kernels
    still use it) is that stream's memory: the allocator then hands it on in that
    stream's order only. Memory of the current stream would go to the current
    stream's next allocation at once, or come from work there that is not done
    with it."""
    cuda = _torch().cuda
    with cuda.stream(stream if isinstance(stream, cuda.Stream) else cuda.ExternalStream(stream.cuda_stream)):
        return wrapper(**{**arguments, "stream": None})


@dataclass
class MXTensor:
    """One quantised copy ([rows, k] E4M3 codes + swizzled E8M0 scales)."""
    data: "object"      # torch.uint8 [rows, ld]
    scale: "object"     # torch.uint8 [mx_scale_bytes(rows, k)]
    rows: int
    k: int
    orient: int         # MX_ROWWISE or MX_COLWISE

    def c_operand(self) -> MXOperandC:
        assert self.data.is_cuda and self.scale.is_cuda, "a product's operands: CUDA tensors"
        return MXOperandC(self.data.data_ptr(), self.scale.data_ptr(), self.rows, self.k,
                          int(self.data.stride(0)), self.orient, 0)


def new_status(device=None):
    """A zeroed device int32 for the kernels' device-side status."""
    torch = _torch()
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def read_status(status) -> int:
    return int(status.item())


def quantize(x, axis: int = MX_BOTH, group_offsets=None, col_capacity: Optional[int] = None, status=None,
             stream=None):
    """MX-quantise a 2-D BF16 (or FP32, no groups) CUDA tensor. Returns
    (row_copy, col_copy), each an MXTensor or None. With ``group_offsets``
    (int64 CUDA tensor [E+1]) the column copy is per-group padded with width
    ``col_capacity``."""
    if stream is not None:
        return _under(stream, quantize, locals())
    torch = _torch()
    assert x.dim() == 2 and x.dtype in (torch.bfloat16, torch.float32) and x.is_cuda and x.stride(1) == 1
    assert x.dtype == torch.bfloat16 or group_offsets is None
    R, C = x.shape
    dev = x.device
    row = col = None
    if axis & MX_ROWWISE:
        row = MXTensor(torch.empty((R, C), dtype=torch.uint8, device=dev),
                       torch.empty(mx_scale_bytes(R, C), dtype=torch.uint8, device=dev), R, C, MX_ROWWISE)
    n_groups = 0
    cap = 0
    if axis & MX_COLWISE:
        if group_offsets is not None:
            n_groups = group_offsets.numel() - 1
            cap = int(col_capacity) if col_capacity is not None else ((R + 127 * n_groups + 127) // 128) * 128
            col = MXTensor(torch.empty((C, cap), dtype=torch.uint8, device=dev),
                           torch.empty(mx_scale_bytes(C, cap), dtype=torch.uint8, device=dev), C, cap, MX_COLWISE)
        else:
            col = MXTensor(torch.empty((C, R), dtype=torch.uint8, device=dev),
                           torch.empty(mx_scale_bytes(C, R), dtype=torch.uint8, device=dev), C, R, MX_COLWISE)
    if x.dtype == torch.float32:
        mx_quantize_f32(x.data_ptr(), 1, R, C, x.stride(0), 0, axis,
                        _ptr(row.data) if row else None, _ptr(row.scale) if row else None,
                        _ptr(col.data) if col else None, _ptr(col.scale) if col else None,
                        _given(status), _stream(stream))
        return row, col
    mx_quantize(x.data_ptr(), R, C, x.stride(0), axis,
                _ptr(row.data) if row else None, _ptr(row.scale) if row else None,
                _ptr(col.data) if col else None, _ptr(col.scale) if col else None,
                _given(group_offsets), n_groups, cap, _given(status), _stream(stream))
    return row, col


def quantize_multi(xs, axis: int = MX_BOTH, status=None, stream=None):
    """MX-quantise up to MX_MAX_MULTI 2-D BF16 CUDA tensors of any shapes in
    one launch. Returns a list of (row_copy, col_copy), one per input, each
    exactly what ``quantize`` gives for that input alone."""
    if stream is not None:
        return _under(stream, quantize_multi, locals())
    torch = _torch()
    outs, descs = [], []
    for x in xs:
        assert x.dim() == 2 and x.dtype == torch.bfloat16 and x.is_cuda
        assert x.numel() == 0 or x.stride(1) == 1
        R, C = x.shape
        dev = x.device
        row = col = None
        if axis & MX_ROWWISE:
            row = MXTensor(torch.empty((R, C), dtype=torch.uint8, device=dev),
                           torch.empty(mx_scale_bytes(R, C), dtype=torch.uint8, device=dev), R, C, MX_ROWWISE)
        if axis & MX_COLWISE:
            col = MXTensor(torch.empty((C, R), dtype=torch.uint8, device=dev),
                           torch.empty(mx_scale_bytes(C, R), dtype=torch.uint8, device=dev), C, R, MX_COLWISE)
        outs.append((row, col))
        ldx = x.stride(0) if x.numel() else C  # an empty matrix's strides carry no pitch
        descs.append(MXQuantTensorC(x.data_ptr(), R, C, ldx,
                                    _ptr(row.data) if row else None, _ptr(row.scale) if row else None,
                                    _ptr(col.data) if col else None, _ptr(col.scale) if col else None))
    mx_quantize_multi(descs, axis, _given(status), _stream(stream))
    return outs


def gemm(mode: int, a: MXTensor, b: MXTensor, out=None, status=None, stream=None, workspace=None):
    """C[M, N] = A . B^T in BF16 (FP32 accumulation). With `workspace` (a CUDA
    uint8 tensor, see gemm_workspace) the GEMM may split its last round."""
    if stream is not None:
        return _under(stream, gemm, locals())
    torch = _torch()
    assert workspace is None or workspace.is_cuda, "workspace: a CUDA tensor"
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=torch.bfloat16, device=a.data.device)
    if workspace is None:
        mx_gemm(mode, a.c_operand(), b.c_operand(), _output(out), out.stride(0), _given(status), _stream(stream))
    else:
        mx_gemm_with_workspace(mode, a.c_operand(), b.c_operand(), _output(out), out.stride(0),
                               workspace.data_ptr() if workspace.numel() else None, workspace.numel(),
                               _given(status), _stream(stream))
    return out


def gemm_workspace(mode: int, a: MXTensor, b: MXTensor):
    """A workspace of the size mx_gemm_with_workspace uses for these operands
    (an empty tensor when the GEMM does not split)."""
    torch = _torch()
    n = mx_gemm_workspace_bytes(mode, a.c_operand(), b.c_operand())
    return torch.empty(n, dtype=torch.uint8, device=a.data.device)


def gemm_multi(problems, status=None, stream=None):
    """Several independent GEMMs (mode, a, b[, out]) in one launch; returns the
    outputs (BF16 [a.rows, b.rows], allocated where not given)."""
    if stream is not None:
        return _under(stream, gemm_multi, locals())
    torch = _torch()
    outs, descs = [], []
    for pr in problems:
        mode, a, b = pr[0], pr[1], pr[2]
        out = pr[3] if len(pr) > 3 and pr[3] is not None else \
            torch.empty((a.rows, b.rows), dtype=torch.bfloat16, device=a.data.device)
        outs.append(out)
        descs.append(MXGemmProblemC(a.c_operand(), b.c_operand(), _output(out), out.stride(0), mode, 0))
    mx_gemm_multi(descs, _given(status), _stream(stream))
    return outs


@dataclass
class MXStacked:
    """Per-expert quantised copies stacked as [E][rows][k] with per-expert
    scale blocks of mx_scale_bytes(rows, k) bytes."""
    data: "object"      # torch.uint8 [E, rows, k]
    scale: "object"     # torch.uint8 [E, mx_scale_bytes(rows, k)]
    rows: int
    k: int
    orient: int

    def c_operand(self) -> MXOperandC:
        assert self.data.is_cuda and self.scale.is_cuda, "a product's operands: CUDA tensors"
        return MXOperandC(self.data.data_ptr(), self.scale.data_ptr(), self.rows, self.k,
                          int(self.data.stride(1)), self.orient, 0)


def quantize_stacked(w, axis: int, status=None, stream=None):
    """Quantise stacked expert weights w[E, N, K] (BF16, or the FP32 master) in
    one batched launch. Returns (row_stack [E][N][K], col_stack [E][K][N]);
    entries None if not asked."""
    if stream is not None:
        return _under(stream, quantize_stacked, locals())
    torch = _torch()
    E, N, K = w.shape
    dev = w.device
    row = col = None
    if axis & MX_ROWWISE:
        row = MXStacked(torch.empty((E, N, K), dtype=torch.uint8, device=dev),
                        torch.empty((E, mx_scale_bytes(N, K)), dtype=torch.uint8, device=dev), N, K, MX_ROWWISE)
    if axis & MX_COLWISE:
        col = MXStacked(torch.empty((E, K, N), dtype=torch.uint8, device=dev),
                        torch.empty((E, mx_scale_bytes(K, N)), dtype=torch.uint8, device=dev), K, N, MX_COLWISE)
    assert w.is_cuda and w.stride(2) == 1 and w.dtype in (torch.bfloat16, torch.float32)
    fn = mx_quantize_f32 if w.dtype == torch.float32 else mx_quantize_batched
    fn(w.data_ptr(), E, N, K, w.stride(1), w.stride(0), axis,
       _ptr(row.data) if row else None, _ptr(row.scale) if row else None,
       _ptr(col.data) if col else None, _ptr(col.scale) if col else None,
       _given(status), _stream(stream))
    return row, col


def grouped_gemm(mode: int, a, b, group_offsets, out=None, status=None, stream=None):
    """Grouped GEMM. fprop/dgrad: a MXTensor [M_total, K] (rows grouped by
    expert), b MXStacked [E][N][K] -> out [M_total, N]. wgrad: a, b grouped
    column copies (MXTensor [N, cap], [Kout, cap]) -> out [E, N, Kout]."""
    if stream is not None:
        return _under(stream, grouped_gemm, locals())
    torch = _torch()
    assert group_offsets.is_cuda, "group_offsets: a CUDA tensor"
    E = group_offsets.numel() - 1
    if out is None:
        if mode == MX_WGRAD:
            out = torch.empty((E, a.rows, b.rows), dtype=torch.bfloat16, device=a.data.device)
        else:
            out = torch.empty((a.rows, b.rows), dtype=torch.bfloat16, device=a.data.device)
    ldc = out.stride(-2)
    mx_grouped_gemm(mode, a.c_operand(), b.c_operand(), group_offsets.data_ptr(), E, _output(out), ldc,
                    _given(status), _stream(stream))
    return out


def grouped_gemm_swiglu(a, b, group_offsets, out=None, status=None, stream=None):
    """Grouped gate_up fprop with SwiGLU in the epilogue: a MXTensor [M_total, K]
    (rows grouped by expert), b MXStacked [E][2F][K] (gate rows first) ->
    out [M_total, F] = silu(gate) * up in BF16."""
    if stream is not None:
        return _under(stream, grouped_gemm_swiglu, locals())
    torch = _torch()
    assert group_offsets.is_cuda, "group_offsets: a CUDA tensor"
    E = group_offsets.numel() - 1
    if out is None:
        out = torch.empty((a.rows, b.rows // 2), dtype=torch.bfloat16, device=a.data.device)
    mx_grouped_gemm_swiglu(a.c_operand(), b.c_operand(), group_offsets.data_ptr(), E, _output(out), out.stride(0),
                           _given(status), _stream(stream))
    return out


def grouped_gemm_swiglu_quantize(a, b, group_offsets, col_capacity: int, out=None, status=None, stream=None):
    """grouped_gemm_swiglu with the output's MX copies written instead of the
    output: returns (row_copy, col_copy) as quantize(output, MX_BOTH,
    group_offsets, col_capacity) would ([M_total, F] and the per-expert padded
    [F, col_capacity]). ``out``: an existing (row_copy, col_copy) pair to fill."""
    if stream is not None:
        return _under(stream, grouped_gemm_swiglu_quantize, locals())
    torch = _torch()
    assert group_offsets.is_cuda, "group_offsets: a CUDA tensor"
    E = group_offsets.numel() - 1
    R, F = a.rows, b.rows // 2
    dev = a.data.device
    if out is None:
        row = MXTensor(torch.empty((R, F), dtype=torch.uint8, device=dev),
                       torch.empty(mx_scale_bytes(R, F), dtype=torch.uint8, device=dev), R, F, MX_ROWWISE)
        col = MXTensor(torch.empty((F, col_capacity), dtype=torch.uint8, device=dev),
                       torch.empty(mx_scale_bytes(F, col_capacity), dtype=torch.uint8, device=dev), F, col_capacity,
                       MX_COLWISE)
    else:
        row, col = out
        assert all(t.is_cuda for c in out for t in (c.data, c.scale)), "out: copies of CUDA tensors"
    mx_grouped_gemm_swiglu_quantize(a.c_operand(), b.c_operand(), group_offsets.data_ptr(), E, _ptr(row.data),
                                    _ptr(row.scale), _ptr(col.data), _ptr(col.scale), col_capacity, _given(status),
                                    _stream(stream))
    return row, col


@dataclass
class FP8Blockwise:
    """E4M3 data [rows, k] with FP32 block multipliers: block 1 -> scale
    [k/128, rows] (1 x 128 blocks), block 128 -> scale [ceil(rows/128), k/128]."""
    data: "object"
    scale: "object"
    rows: int
    k: int
    block: int


def quantize_fp8_blockwise(x, block: int, status=None, stream=None) -> FP8Blockwise:
    """DeepSeek-V3 blockwise FP8 quantisation of a 2-D BF16 CUDA tensor."""
    if stream is not None:
        return _under(stream, quantize_fp8_blockwise, locals())
    torch = _torch()
    assert x.dim() == 2 and x.dtype == torch.bfloat16 and x.is_cuda and x.stride(1) == 1
    R, C = x.shape
    data = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    shape = (C // 128, R) if block == 1 else ((R + 127) // 128, C // 128)
    scale = torch.empty(shape, dtype=torch.float32, device=x.device)
    mx_quantize_fp8_blockwise(x.data_ptr(), R, C, x.stride(0), block, data.data_ptr(), scale.data_ptr(),
                              _given(status), _stream(stream))
    return FP8Blockwise(data, scale, R, C, block)


def gemm_fp8_blockwise(a: FP8Blockwise, b: FP8Blockwise, out=None, status=None, stream=None):
    """C[M, N] = A . B^T for an activation (block 1) and a weight (block 128)."""
    if stream is not None:
        return _under(stream, gemm_fp8_blockwise, locals())
    torch = _torch()
    assert a.block == 1 and b.block == 128 and a.k == b.k
    assert all(t.is_cuda for t in (a.data, a.scale, b.data, b.scale)), "a product's operands: CUDA tensors"
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=torch.bfloat16, device=a.data.device)
    mx_gemm_fp8_blockwise(a.data.data_ptr(), a.scale.data_ptr(), a.rows, b.data.data_ptr(), b.scale.data_ptr(),
                          b.rows, a.k, _output(out), out.stride(0), _given(status), _stream(stream))
    return out


# ---------------------------------------------------------------------------
# Current-scaling variant (one FP32 scale per tensor or per expert)
# ---------------------------------------------------------------------------

CURRENT_FORMAT_MAX = 448.0


def current_amax(x, status=None, stream=None):
    """amax of a 2-D BF16 tensor ([1] FP32) or of each matrix of a 3-D stack ([E])."""
    if stream is not None:
        return _under(stream, current_amax, locals())
    torch = _torch()
    xs = x if x.dim() == 3 else x.unsqueeze(0)
    assert xs.dtype == torch.bfloat16 and xs.is_cuda and xs.stride(2) == 1
    E, R, C = xs.shape
    amax = torch.empty(E, dtype=torch.float32, device=x.device)
    mx_current_amax(xs.data_ptr(), E, R, C, xs.stride(1), xs.stride(0), amax.data_ptr(), _given(status), _stream(stream))
    return amax


def quantize_current(x, axis: int = MX_BOTH, amax=None, format_max: float = CURRENT_FORMAT_MAX, group_offsets=None,
                     col_capacity: Optional[int] = None, status=None, stream=None):
    """Current-scaling quantisation of a 2-D BF16 tensor (or a 3-D stack, one
    scale per matrix). amax: FP32 [batch] (computed here when None). Returns
    (row_copy, col_copy); each copy's `scale` is the FP32 scale tensor [batch]
    (the same tensor for both copies)."""
    if stream is not None:
        return _under(stream, quantize_current, locals())
    torch = _torch()
    stacked = x.dim() == 3
    xs = x if stacked else x.unsqueeze(0)
    assert x.is_cuda and (amax is None or amax.is_cuda), "needs CUDA tensors"
    E, R, C = xs.shape
    dev = x.device
    if amax is None:
        amax = current_amax(x, status=status, stream=stream)
    scale = torch.empty(E, dtype=torch.float32, device=dev)
    u8 = dict(dtype=torch.uint8, device=dev)
    row = col = None
    n_groups, cap = 0, 0
    if axis & MX_ROWWISE:
        d = torch.empty((E, R, C), **u8)
        row = (MXStacked(d, scale, R, C, MX_ROWWISE) if stacked else MXTensor(d[0], scale, R, C, MX_ROWWISE))
    if axis & MX_COLWISE:
        if group_offsets is not None:
            assert not stacked
            n_groups = group_offsets.numel() - 1
            cap = int(col_capacity) if col_capacity is not None else ((R + 127 * n_groups + 127) // 128) * 128
            col = MXTensor(torch.empty((C, cap), **u8), scale, C, cap, MX_COLWISE)
        else:
            d = torch.empty((E, C, R), **u8)
            col = (MXStacked(d, scale, C, R, MX_COLWISE) if stacked else MXTensor(d[0], scale, C, R, MX_COLWISE))
    mx_quantize_current(xs.data_ptr(), E, R, C, xs.stride(1), xs.stride(0), axis, amax.data_ptr(), float(format_max),
                        _ptr(row.data) if row else None, _ptr(col.data) if col else None, scale.data_ptr(),
                        _given(group_offsets), n_groups, cap, _given(status), _stream(stream))
    return row, col


def gemm_current(mode: int, a, b, out=None, status=None, stream=None):
    """C[M, N] = (A . B^T) * s_a * s_b in BF16 for current-scaled operands."""
    if stream is not None:
        return _under(stream, gemm_current, locals())
    torch = _torch()
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=torch.bfloat16, device=a.data.device)
    mx_gemm_current(mode, a.c_operand(), b.c_operand(), _output(out), out.stride(0), _given(status), _stream(stream))
    return out


def gemm_current_multi(problems, status=None, stream=None):
    """Several independent current-scaled GEMMs (mode, a, b[, out]) in one
    launch; returns the outputs (BF16 [a.rows, b.rows], allocated where not
    given)."""
    if stream is not None:
        return _under(stream, gemm_current_multi, locals())
    torch = _torch()
    outs, descs = [], []
    for pr in problems:
        mode, a, b = pr[0], pr[1], pr[2]
        out = pr[3] if len(pr) > 3 and pr[3] is not None else \
            torch.empty((a.rows, b.rows), dtype=torch.bfloat16, device=a.data.device)
        outs.append(out)
        descs.append(MXGemmProblemC(a.c_operand(), b.c_operand(), _output(out), out.stride(0), mode, 0))
    mx_gemm_current_multi(descs, _given(status), _stream(stream))
    return outs


def grouped_gemm_current(mode: int, a, b, group_offsets, out=None, status=None, stream=None):
    """Grouped GEMM on current-scaled operands (layouts as grouped_gemm; the
    stacked weights carry one scale per expert)."""
    if stream is not None:
        return _under(stream, grouped_gemm_current, locals())
    torch = _torch()
    assert group_offsets.is_cuda, "group_offsets: a CUDA tensor"
    E = group_offsets.numel() - 1
    if out is None:
        shape = (E, a.rows, b.rows) if mode == MX_WGRAD else (a.rows, b.rows)
        out = torch.empty(shape, dtype=torch.bfloat16, device=a.data.device)
    mx_grouped_gemm_current(mode, a.c_operand(), b.c_operand(), group_offsets.data_ptr(), E, _output(out),
                            out.stride(-2), _given(status), _stream(stream))
    return out


# ---------------------------------------------------------------------------
# Operators around the products of a training step
# ---------------------------------------------------------------------------

def _dtype(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return MX_BF16
    assert t.dtype == torch.float32, f"needs BF16 or FP32, got {t.dtype}"
    return MX_F32


@dataclass
class AdamWState:
    """AdamW's two moments of one tensor. bits 32: FP32 tensors like it. bits 8:
    code tensors of its numel (exp_avg: E4M3 as float8_e4m3fn or uint8;
    exp_avg_sq: uint8) with one FP32 scale per MX_ADAMW_STATE_BLOCK elements."""
    bits: int
    exp_avg: "object"
    exp_avg_sq: "object"
    exp_avg_scale: "object" = None
    exp_avg_sq_scale: "object" = None


def adamw_state(param, bits: int = 32) -> AdamWState:
    """The zero state of a parameter, before its first step."""
    torch = _torch()
    assert bits in (32, 8)
    if bits == 32:
        return AdamWState(32, torch.zeros_like(param, dtype=torch.float32), torch.zeros_like(param, dtype=torch.float32))
    n = param.numel()
    blocks = (n + MX_ADAMW_STATE_BLOCK - 1) // MX_ADAMW_STATE_BLOCK
    u8 = dict(dtype=torch.uint8, device=param.device)
    f32 = dict(dtype=torch.float32, device=param.device)
    return AdamWState(8, torch.zeros(n, **u8), torch.zeros(n, **u8), torch.zeros(blocks, **f32),
                      torch.zeros(blocks, **f32))


_ADAMW_TENSOR = "6Qqd2i"  # mx_adamw_tensor


def adamw_step(params, grads, states, lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.0,
               step: int = 1, grad_scale=None, seed: Optional[int] = None, status=None, stream=None) -> None:
    """One AdamW step, in place, over all tensors in one launch (per 448).

    params: contiguous FP32 CUDA tensors; grads: contiguous, FP32 or BF16, each
    of its parameter's numel; states: one AdamWState each, all of the same bits.
    weight_decay: one value, or one per tensor. step counts from 1. grad_scale:
    a CUDA FP32 tensor of one element that multiplies every gradient; where it
    is not finite the step changes nothing (status 5). seed: with 8-bit states,
    the second moment's random rounding; a new one every step (the same one would
    round an element the same way every time, and its moment would stand still).
    Default: the step count."""
    torch = _torch()
    n = len(params)
    assert len(grads) == n and len(states) == n, "one gradient and one state per parameter"
    if n == 0:
        return
    f32, bf16 = torch.float32, torch.bfloat16
    bits = states[0].bits
    decay = weight_decay if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
    # Attribute by attribute over all tensors rather than tensor by tensor: a
    # step over many small tensors is bound by this function.
    T = torch.Tensor
    tensors = [*params, *grads, *[s.exp_avg for s in states], *[s.exp_avg_sq for s in states]]
    size, ptr, dtype = (list(map(f, tensors)) for f in (T.numel, T.data_ptr, T.dtype.__get__))
    kinds = set(dtype[n:2 * n])
    assert len(decay) == n and all([s.bits == bits for s in states]), "all states of one call have the same bits"
    assert set(dtype[:n]) == {f32}, "parameters: FP32"
    assert kinds <= {f32, bf16}, "gradients: FP32 or BF16"
    assert size == size[:n] * 4, "gradients and states: of the parameters' sizes"
    if bits == 8:
        scales = [*[s.exp_avg_scale for s in states], *[s.exp_avg_sq_scale for s in states]]
        assert {t.itemsize for t in set(dtype[2 * n:])} == {1}, "8-bit states: one byte an element"
        assert set(map(T.dtype.__get__, scales)) == {f32}, "scales: FP32"
        assert all([k >= (m + MX_ADAMW_STATE_BLOCK - 1) // MX_ADAMW_STATE_BLOCK
                    for k, m in zip(map(T.numel, scales), size[2 * n:])]), "scales: one per block"
        tensors += scales
        ptr += map(T.data_ptr, scales)
    else:
        assert set(dtype[2 * n:]) == {f32}, "32-bit states: FP32"
        ptr += [0] * (2 * n)
    assert all(map(T.is_contiguous, tensors)) and all(map(T.is_cuda.__get__, tensors)), "contiguous CUDA tensors"
    if grad_scale is not None:
        assert grad_scale.dtype is f32 and grad_scale.is_cuda and grad_scale.numel() == 1
    g32 = [0] * n if kinds == {bf16} else [int(t is f32) for t in dtype[n:2 * n]]
    rows = zip(*[ptr[k * n:(k + 1) * n] for k in range(6)], size, decay, g32, [0] * n)
    hyper = MXAdamWHyperC(lr, betas[0], betas[1], eps, step, (step if seed is None else seed) & 0xFFFFFFFF, 0)
    mx_adamw_step(struct.pack(_ADAMW_TENSOR * n, *itertools.chain.from_iterable(rows)), n, bits, hyper, _ptr(grad_scale),
                  _given(status), _stream(stream))


def _rows(t) -> int:
    """Pitch of a 2-D matrix with contiguous rows."""
    R, C = t.shape
    p, q = t.stride()
    assert t.is_cuda and (q == 1 or C <= 1), "needs 2-D CUDA tensors with contiguous rows"
    return p if R > 1 else C


def _params(weight, bias, cols) -> int:
    """The one dtype of a norm's weight and bias."""
    dtype = MX_F32
    for p in (weight, bias):
        if p is not None:
            assert p.is_cuda and p.is_contiguous() and p.numel() == cols, "weight and bias: contiguous, one entry per column"
            dtype = _dtype(p)
    assert weight is None or bias is None or weight.dtype == bias.dtype, "weight and bias have the same dtype"
    return dtype


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, center: bool = True, out=None, stats: bool = True,
               status=None, stream=None):
    """Layer norm of each row of x (2-D, BF16 or FP32, any row pitch), or with
    center=False the root-mean-square norm. Returns (y, mean, rstd): y in x's
    dtype, the FP32 row statistics for layer_norm_backward (mean None with
    center=False, both None with stats=False)."""
    if stream is not None:
        return _under(stream, layer_norm, locals())
    torch = _torch()
    R, C = x.shape
    dev = x.device
    dtype, pd, ldx, ldy = _dtype(x), _params(weight, bias, C), _rows(x), C
    if out is None:
        out = torch.empty((R, C), dtype=x.dtype, device=dev)
    else:
        assert out.dtype == x.dtype and out.shape == x.shape
        ldy = _rows(out)
    mean = torch.empty(R, dtype=torch.float32, device=dev) if stats and center else None
    rstd = torch.empty(R, dtype=torch.float32, device=dev) if stats else None
    mx_layer_norm(x.data_ptr(), ldx, _ptr(weight), _ptr(bias), pd, R, C, eps, int(center), dtype, out.data_ptr(), ldy,
                  _ptr(mean), _ptr(rstd), _given(status), _stream(stream))
    return out, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, center: bool = True, param_grads: bool = True, status=None,
                        stream=None):
    """Gradients of layer_norm: (dx in x's dtype, dweight FP32, dbias FP32; the
    two None with param_grads=False). mean and rstd are layer_norm's."""
    if stream is not None:
        return _under(stream, layer_norm_backward, locals())
    torch = _torch()
    R, C = x.shape
    dev = x.device
    assert dy.shape == x.shape and dy.dtype == x.dtype
    for t in (rstd, mean) if center else (rstd,):
        assert t.is_cuda and t.dtype == torch.float32 and t.is_contiguous() and t.numel() == R, \
            "mean and rstd: contiguous FP32 CUDA tensors, one entry per row"
    pd = _params(weight, None, C)
    dx = torch.empty((R, C), dtype=x.dtype, device=dev)
    dw = db = ws = None
    need = 0
    if param_grads:
        dw = torch.empty(C, dtype=torch.float32, device=dev)
        db = torch.empty(C, dtype=torch.float32, device=dev)
        need = mx_layer_norm_backward_workspace_bytes(R, C)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    mx_layer_norm_backward(dy.data_ptr(), _rows(dy), x.data_ptr(), _rows(x), _ptr(weight), pd,
                           _ptr(mean) if center else None, rstd.data_ptr(), R, C, int(center), _dtype(x), dx.data_ptr(),
                           C, _ptr(dw), _ptr(db), _ptr(ws), need, _given(status), _stream(stream))
    return dx, dw, db


def gemm_epilogue(mode: int, a: MXTensor, b: MXTensor, bias=None, act: str = "none", residual=None,
                  keep_preact: bool = False, out=None, preact=None, status=None, stream=None):
    """out = act(A . B^T + bias) + residual in BF16, from the FP32 accumulators.
    bias: [N] FP32 or BF16; residual: BF16 [M, N] (may be ``out``); act: one of
    ACTIVATIONS. Returns (out, z): z the BF16 pre-activation for
    epilogue_backward with keep_preact (or a ``preact`` tensor to fill), else None."""
    if stream is not None:
        return _under(stream, gemm_epilogue, locals())
    torch = _torch()
    M, N = a.rows, b.rows
    dev = a.data.device
    bf16 = torch.bfloat16

    def pitch(t):
        assert t.dtype == bf16 and t.shape == (M, N), "out, residual and preact: BF16 [M, N]"
        return _rows(t)

    ldc, ldr, ldz = N, 0 if residual is None else pitch(residual), N
    if out is None:
        out = torch.empty((M, N), dtype=bf16, device=dev)
    else:
        ldc = pitch(out)
    if preact is not None:
        ldz = pitch(preact)
    elif keep_preact:
        preact = torch.empty((M, N), dtype=bf16, device=dev)
    bd = MX_F32
    if bias is not None:
        assert bias.is_cuda and bias.is_contiguous() and bias.numel() == N, "bias: contiguous, one entry per column"
        bd = _dtype(bias)
    e = MXEpilogueC(_ptr(bias), _ptr(residual), _ptr(preact), ldr, ldz, bd, ACTIVATIONS[act])
    mx_gemm_epilogue(mode, a.c_operand(), b.c_operand(), e, out.data_ptr(), ldc, _given(status), _stream(stream))
    return out, preact


def epilogue_backward(dy, preact, act: str = "none", bias_grad: bool = True, dz=None, status=None, stream=None):
    """Gradient of gemm_epilogue's epilogue: (dz BF16 [M, N], dbias FP32 [N] or
    None). preact: gemm_epilogue's z (unused, may be None, with act "none")."""
    if stream is not None:
        return _under(stream, epilogue_backward, locals())
    torch = _torch()
    assert dy.dtype == torch.bfloat16
    M, N = dy.shape
    a = ACTIVATIONS[act]
    assert a == MX_ACT_NONE or (preact.dtype == torch.bfloat16 and preact.shape == dy.shape), "preact: BF16, of dy's shape"
    lddz = N
    if dz is None:
        dz = torch.empty((M, N), dtype=torch.bfloat16, device=dy.device)
    else:
        assert dz.dtype == torch.bfloat16 and dz.shape == dy.shape
        lddz = _rows(dz)
    dbias = ws = None
    need = 0
    if bias_grad:
        dbias = torch.empty(N, dtype=torch.float32, device=dy.device)
        need = mx_epilogue_backward_workspace_bytes(M, N)
        ws = torch.empty(need, dtype=torch.uint8, device=dy.device) if need else None
    mx_epilogue_backward(dy.data_ptr(), _rows(dy), _ptr(preact), 0 if preact is None else _rows(preact), M, N, a,
                         dz.data_ptr(), lddz, _ptr(dbias), _ptr(ws), need, _given(status), _stream(stream))
    return dz, dbias


@dataclass
class Routing:
    """What router_forward returns."""
    indices: "object"        # int32 [T, top_k], -1: no choice
    weights: "object"        # FP32 [T, top_k]
    counts: "object"         # int64 [E]
    group_offsets: "object"  # int64 [E + 1], the grouped calls' offsets
    load: "object"           # FP32 [sequences, E], for router_backward
    loss: "object"           # FP32 [1]


def router_forward(logits, top_k: int, tokens_per_seq: Optional[int] = None, token_mask=None, normalize: bool = False,
                   coef: float = 1.0, status=None, stream=None) -> Routing:
    """Routes logits [T, E] (FP32 or BF16, any row pitch): the top_k experts of
    each token (ties to the lowest), their softmax weights (divided by their sum
    with normalize), the per-expert counts and group offsets, and the balance
    loss, averaged over sequences of tokens_per_seq tokens (default: one
    sequence). token_mask: bool or uint8 [T], false: left out."""
    if stream is not None:
        return _under(stream, router_forward, locals())
    torch = _torch()
    T, E = logits.shape
    dev = logits.device
    seq = max(T, 1) if tokens_per_seq is None else tokens_per_seq
    assert seq >= 1 and 1 <= top_k <= E
    mask = _mask(token_mask, T)
    empty, f32, i64 = torch.empty, torch.float32, torch.int64
    indices = empty((T, top_k), dtype=torch.int32, device=dev)
    weights = empty((T, top_k), dtype=f32, device=dev)
    counts = empty(E, dtype=i64, device=dev)
    offsets = empty(E + 1, dtype=i64, device=dev)
    load = empty(((T + seq - 1) // seq, E), dtype=f32, device=dev)
    loss = empty(1, dtype=f32, device=dev)
    need = mx_router_workspace_bytes(T, seq, E)
    ws = empty(need, dtype=torch.uint8, device=dev)
    mx_router_forward(logits.data_ptr(), _rows(logits), _dtype(logits), mask, T, seq, E, top_k, int(normalize), coef,
                      indices.data_ptr(), weights.data_ptr(), counts.data_ptr(), offsets.data_ptr(), load.data_ptr(),
                      loss.data_ptr(), ws.data_ptr(), need, _given(status), _stream(stream))
    return Routing(indices, weights, counts, offsets, load, loss)


def _mask(token_mask, tokens) -> Optional[int]:
    if token_mask is None:
        return None
    torch = _torch()
    assert token_mask.dtype in (torch.bool, torch.uint8) and token_mask.is_cuda and token_mask.is_contiguous()
    assert token_mask.numel() == tokens, "token_mask: one entry per token"
    return token_mask.data_ptr()


def router_backward(logits, indices, load, dweights=None, dloss=None, tokens_per_seq: Optional[int] = None,
                    token_mask=None, normalize: bool = False, status=None, stream=None):
    """dlogits (logits' dtype) from dweights (FP32 [T, top_k] or None) and dloss
    (FP32 [1] on the device, or None); indices, load, tokens_per_seq, token_mask
    and normalize as in router_forward."""
    if stream is not None:
        return _under(stream, router_backward, locals())
    torch = _torch()
    T, E = logits.shape
    top_k = indices.shape[1]
    seq = max(T, 1) if tokens_per_seq is None else tokens_per_seq
    f32 = torch.float32
    assert indices.is_cuda and load.is_cuda and (dweights is None or dweights.is_cuda), "CUDA tensors"
    assert indices.dtype == torch.int32 and indices.is_contiguous() and indices.shape[0] == T
    assert load.dtype == f32 and load.is_contiguous() and load.shape == ((T + seq - 1) // seq, E)
    assert dweights is None or (dweights.dtype == f32 and dweights.is_contiguous() and dweights.shape == indices.shape)
    assert dloss is None or (dloss.dtype == f32 and dloss.is_cuda and dloss.numel() == 1)
    dx = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    mx_router_backward(logits.data_ptr(), _rows(logits), _dtype(logits), _mask(token_mask, T), T, seq, E, top_k,
                       int(normalize), indices.data_ptr(), load.data_ptr(), _ptr(dweights), _ptr(dloss), dx.data_ptr(),
                       E, _given(status), _stream(stream))
    return dx


# ---------------------------------------------------------------------------
# The gated feed-forward block's wrappers: a module of their own, loaded when one
# of them is first asked for
# ---------------------------------------------------------------------------

_GATED_BLOCK = ("AddNorm", "AddNormGrads", "add_norm_quantize", "add_norm_backward", "gemm_gated", "gated_quantize",
                "gated_backward_quantize")


_gated_block = None


def __getattr__(name):
    global _gated_block
    if name in _GATED_BLOCK:
        if _gated_block is None:
            from . import gated_block as _gated_block
        return getattr(_gated_block, name)
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted([*globals(), *_GATED_BLOCK])
