"""Wrappers of the gated feed-forward block's calls for torch tensors (reached as
the package's own names): the residual's addition with the norm, the product with
its gate, and the gate's quantising calls, forward and backward. Argument
marshalling only, as in the package."""

from __future__ import annotations

import functools
from dataclasses import dataclass
from typing import Optional

import torch

import mxfp8_block_scaled_gb300 as mx

# A small call costs what its wrapper does on the host, so the wrappers look little up:
# sizes of scale buffers are asked for once, a matrix's checks are one call.
_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8
_DTYPE = {_BF16: mx.MX_BF16, _F32: mx.MX_F32}
_scale_bytes = functools.lru_cache(maxsize=1024)(mx.mx_scale_bytes)
_norm_workspace = functools.lru_cache(maxsize=1024)(mx.mx_add_norm_backward_workspace_bytes)


def _matrix(t, rows, cols, dtype, what) -> int:
    """Pitch of a [rows, cols] matrix of contiguous rows."""
    assert t.dtype is dtype and t.shape == (rows, cols), what
    p, q = t.stride()
    assert t.is_cuda and (q == 1 or cols <= 1), "needs 2-D CUDA tensors with contiguous rows"
    return p if rows > 1 else cols


def _copy(rows, k, orient, dev) -> mx.MXTensor:
    empty = torch.empty
    return mx.MXTensor(empty((rows, k), dtype=_U8, device=dev), empty(_scale_bytes(rows, k), dtype=_U8, device=dev), rows, k, orient)


def _copies(axis, rows, cols, dev, group_offsets=None, col_capacity=None):
    """The copies of a [rows, cols] matrix that ``axis`` asks for, as quantize
    lays them out, and the raw call's arguments for them: (row, col, pointers,
    n_groups, capacity)."""
    assert 0 <= axis <= mx.MX_BOTH, "axis: MX_ROWWISE, MX_COLWISE, MX_BOTH"
    n_groups, cap, width = 0, 0, rows
    if group_offsets is not None:
        assert group_offsets.is_cuda and group_offsets.dtype == torch.int64 and group_offsets.is_contiguous(), \
            "group_offsets: int64 CUDA tensor"
        n_groups = group_offsets.numel() - 1
        cap = width = int(col_capacity) if col_capacity is not None else ((rows + 127 * n_groups + 127) // 128) * 128
    row = col = rd = rs = cd = cs = None
    if axis & mx.MX_ROWWISE:
        row = _copy(rows, cols, mx.MX_ROWWISE, dev)
        rd, rs = row.data.data_ptr(), row.scale.data_ptr()
    if axis & mx.MX_COLWISE:
        col = _copy(cols, width, mx.MX_COLWISE, dev)
        cd, cs = col.data.data_ptr(), col.scale.data_ptr()
    return row, col, (rd, rs, cd, cs), n_groups, cap


@dataclass
class AddNorm:
    """add_norm_quantize's outputs: the sum, the FP32 row statistic, the norm's
    output as MX copies and in BF16 (None where not asked for)."""
    sum: "object"
    rstd: "object"
    row: Optional[mx.MXTensor]
    col: Optional[mx.MXTensor]
    y: "object" = None


@dataclass
class AddNormGrads:
    """add_norm_backward's outputs: dx (the gradient of x and of the residual
    alike, in the stream's dtype), dweight (FP32), dx's MX copies."""
    dx: "object"
    dweight: "object"
    row: Optional[mx.MXTensor]
    col: Optional[mx.MXTensor]


def add_norm_quantize(x, residual=None, weight=None, eps: float = 1e-5, axis: int = mx.MX_BOTH, keep_output: bool = False,
                      stats: bool = True, out=None, status=None, stream=None) -> AddNorm:
    """Adds the residual stream to x (2-D BF16; residual BF16 or FP32, or None)
    and takes the root-mean-square norm of the sum, whose MX copies (``axis``; 0:
    none) are what the next products read. ``out``: where the sum goes (of the
    residual's dtype; may be the residual itself); without a residual and ``out``
    the sum is x. keep_output: the norm's output in BF16 too (a router's input).
    Any row pitch of whole 16-byte pieces."""
    if stream is not None:
        return mx._under(stream, add_norm_quantize, locals())
    R, C = x.shape
    dev, empty = x.device, torch.empty
    ldx = _matrix(x, R, C, _BF16, "x: BF16")
    st, dt, ldr, lds = _BF16, mx.MX_BF16, 0, 0
    if residual is not None:
        st = residual.dtype
        dt, ldr = _DTYPE.get(st), _matrix(residual, R, C, st, "the residual has x's shape")
        assert dt is not None, f"residual: BF16 or FP32, got {st}"
        if out is None:
            out, lds = empty((R, C), dtype=st, device=dev), C
    if lds == 0 and out is not None:
        lds = _matrix(out, R, C, st, "out: x's shape, the residual's dtype")
    row, col, pointers, _, _ = _copies(axis, R, C, dev)
    y = empty((R, C), dtype=_BF16, device=dev) if keep_output else None
    rstd = empty(R, dtype=_F32, device=dev) if stats else None
    mx.mx_add_norm_quantize(x.data_ptr(), ldx, mx._ptr(residual), ldr, dt, mx._ptr(weight), mx._params(weight, None, C), R, C, eps, axis,
                            mx._ptr(out), lds, mx._ptr(y), C, mx._ptr(rstd), *pointers, mx._given(status), mx._stream(None))
    return AddNorm(x if out is None else out, rstd, row, col, y)


def add_norm_backward(dy, sum, weight, rstd, dsum=None, axis: int = 0, weight_grad: bool = True, out=None, status=None,
                      stream=None) -> AddNormGrads:
    """Gradients of add_norm_quantize: dy (BF16) is the norm output's gradient,
    dsum (of sum's dtype, or None) the residual stream's; sum and rstd are the
    forward call's. ``axis``: MX copies of dx too (the dY of the product that
    wrote x). ``out``: where dx goes (may be dsum itself)."""
    if stream is not None:
        return mx._under(stream, add_norm_backward, locals())
    R, C = sum.shape
    dev, st, empty = sum.device, sum.dtype, torch.empty
    dt = _DTYPE.get(st)
    assert dt is not None, f"sum: BF16 or FP32, got {st}"
    lds, lddy = _matrix(sum, R, C, st, "sum"), _matrix(dy, R, C, _BF16, "dy: BF16, of sum's shape")
    assert rstd.is_cuda and rstd.dtype is _F32 and rstd.is_contiguous() and rstd.numel() == R, "rstd: FP32, one per row"
    ldd = 0 if dsum is None else _matrix(dsum, R, C, st, "dsum: sum's dtype and shape")
    if out is None:
        out, ldo = empty((R, C), dtype=st, device=dev), C
    else:
        ldo = _matrix(out, R, C, st, "out: sum's dtype and shape")
    row, col, pointers, _, _ = _copies(axis, R, C, dev)
    dweight, ws, nbytes = None, None, 0
    if weight_grad:
        dweight = empty(C, dtype=_F32, device=dev)
        nbytes = _norm_workspace(R, C)
        ws = empty(nbytes, dtype=_U8, device=dev)
    mx.mx_add_norm_backward(dy.data_ptr(), lddy, sum.data_ptr(), lds, mx._ptr(dsum), ldd, dt, mx._ptr(weight),
                            mx._params(weight, None, C), rstd.data_ptr(), R, C, axis, out.data_ptr(), ldo, mx._ptr(dweight),
                            *pointers, mx._ptr(ws) if nbytes else None, nbytes, mx._given(status), mx._stream(None))
    return AddNormGrads(out, dweight, row, col)


def gemm_gated(a: mx.MXTensor, gate: mx.MXTensor, up: mx.MXTensor, act: str = "silu", keep_preact: bool = False, out=None,
               status=None, stream=None):
    """act(A . gate^T) * (A . up^T) in BF16 [M, F] from row copies of the tokens
    and of the two weights. Returns (out, gate_up): with keep_preact the two
    products side by side, BF16 [M, 2F], for gated_backward_quantize, else None."""
    if stream is not None:
        return mx._under(stream, gemm_gated, locals())
    M, F, act = a.rows, gate.rows, mx.ACTIVATIONS[act]
    dev, empty = a.data.device, torch.empty
    if out is None:
        out, ldc = empty((M, F), dtype=_BF16, device=dev), F
        assert out.is_cuda, "needs CUDA tensors"
    else:
        ldc = _matrix(out, M, F, _BF16, "out: BF16 [M, F]")
    pre = empty((M, 2 * F), dtype=_BF16, device=dev) if keep_preact else None
    mx.mx_gemm_gated(a.c_operand(), gate.c_operand(), up.c_operand(), act, out.data_ptr(), ldc, mx._ptr(pre), 2 * F,
                     mx._given(status), mx._stream(None))
    return out, pre


def gated_quantize(gate_up, act: str = "silu", axis: int = mx.MX_BOTH, group_offsets=None, col_capacity: Optional[int] = None,
                   status=None, stream=None):
    """MX copies (row, col) of h = act(gate) * up from gate_up = [gate | up], BF16
    [rows, 2F]: what the down projection reads. ``group_offsets``, ``col_capacity``:
    the column copy in the experts' segments, as quantize's (the row copy does not
    depend on them)."""
    if stream is not None:
        return mx._under(stream, gated_quantize, locals())
    R, F = gate_up.shape
    ld = _matrix(gate_up, R, F, _BF16, "gate_up: BF16 [rows, 2F]")
    assert F % 2 == 0, "gate_up: BF16 [rows, 2F]"
    F //= 2
    row, col, pointers, n_groups, cap = _copies(axis, R, F, gate_up.device, group_offsets, col_capacity)
    mx.mx_gated_quantize(gate_up.data_ptr(), ld, R, F, mx.ACTIVATIONS[act], axis, *pointers, mx._given(group_offsets), n_groups, cap,
                         mx._given(status), mx._stream(None))
    return row, col


def gated_backward_quantize(dh, gate_up, act: str = "silu", axis: int = mx.MX_BOTH, group_offsets=None,
                            col_capacity: Optional[int] = None, status=None, stream=None):
    """MX copies (row, col) of [dgate | dup], [rows, 2F], from dh (BF16 [rows, F],
    the down projection's dgrad) and gate_up (BF16 [rows, 2F], gemm_gated's or
    grouped_gemm's): the dY of the two projections' dgrad and wgrad."""
    if stream is not None:
        return mx._under(stream, gated_backward_quantize, locals())
    R, F = dh.shape
    lddh = _matrix(dh, R, F, _BF16, "dh: BF16 [rows, F]")
    ld = _matrix(gate_up, R, 2 * F, _BF16, "gate_up: BF16 [rows, 2F]")
    row, col, pointers, n_groups, cap = _copies(axis, R, 2 * F, dh.device, group_offsets, col_capacity)
    mx.mx_gated_backward_quantize(dh.data_ptr(), lddh, gate_up.data_ptr(), ld, R, F, mx.ACTIVATIONS[act], axis, *pointers,
                                  mx._given(group_offsets), n_groups, cap, mx._given(status), mx._stream(None))
    return row, col
