"""Wrappers of the gated feed-forward block's calls for torch tensors (reached as
the package's own names): the residual's addition with the norm, the product with
its gate, and the gate's quantising calls, forward and backward. Argument
marshalling only, as in the package."""

from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import mxfp8_block_scaled_gb300 as mx


def _copy(rows, k, orient, dev) -> mx.MXTensor:
    torch = mx._torch()
    return mx.MXTensor(torch.empty((rows, k), dtype=torch.uint8, device=dev),
                       torch.empty(mx.mx_scale_bytes(rows, k), dtype=torch.uint8, device=dev), rows, k, orient)


def _copies(axis, rows, cols, dev, group_offsets=None, col_capacity=None):
    """The copies of a [rows, cols] matrix that ``axis`` asks for, as quantize
    lays them out, and the raw call's arguments for them: (row, col, pointers,
    n_groups, capacity)."""
    assert 0 <= axis <= mx.MX_BOTH, "axis: MX_ROWWISE, MX_COLWISE, MX_BOTH"
    row = _copy(rows, cols, mx.MX_ROWWISE, dev) if axis & mx.MX_ROWWISE else None
    col, n_groups, cap = None, 0, 0
    if group_offsets is not None:
        torch = mx._torch()
        assert group_offsets.is_cuda and group_offsets.dtype == torch.int64 and group_offsets.is_contiguous(), \
            "group_offsets: int64 CUDA tensor"
        n_groups = group_offsets.numel() - 1
        cap = int(col_capacity) if col_capacity is not None else ((rows + 127 * n_groups + 127) // 128) * 128
    if axis & mx.MX_COLWISE:
        col = _copy(cols, cap if group_offsets is not None else rows, mx.MX_COLWISE, dev)
    pointers = [p for c in (row, col) for p in ((None, None) if c is None else (c.data.data_ptr(), c.scale.data_ptr()))]
    return row, col, pointers, n_groups, cap


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
    torch = mx._torch()
    R, C = x.shape
    dev = x.device
    assert x.dtype == torch.bfloat16, "x: BF16"
    ldx = mx._rows(x)
    sd, ldr = (mx.MX_BF16, 0) if residual is None else (mx._dtype(residual), mx._rows(residual))
    assert residual is None or residual.shape == x.shape, "the residual has x's shape"
    if out is None and residual is not None:
        out = torch.empty((R, C), dtype=residual.dtype, device=dev)
    lds = 0
    if out is not None:
        assert out.shape == x.shape and out.dtype == (torch.bfloat16 if residual is None else residual.dtype), \
            "out: x's shape, the residual's dtype"
        lds = mx._rows(out)
    row, col, pointers, _, _ = _copies(axis, R, C, dev)
    y = torch.empty((R, C), dtype=torch.bfloat16, device=dev) if keep_output else None
    rstd = torch.empty(R, dtype=torch.float32, device=dev) if stats else None
    mx.mx_add_norm_quantize(x.data_ptr(), ldx, mx._ptr(residual), ldr, sd, mx._ptr(weight), mx._params(weight, None, C), R, C, eps, axis,
                         mx._ptr(out), lds, mx._ptr(y), C, mx._ptr(rstd), *pointers, mx._ptr(status), mx._stream(stream))
    return AddNorm(x if out is None else out, rstd, row, col, y)


def add_norm_backward(dy, sum, weight, rstd, dsum=None, axis: int = 0, weight_grad: bool = True, out=None, status=None,
                      stream=None) -> AddNormGrads:
    """Gradients of add_norm_quantize: dy (BF16) is the norm output's gradient,
    dsum (of sum's dtype, or None) the residual stream's; sum and rstd are the
    forward call's. ``axis``: MX copies of dx too (the dY of the product that
    wrote x). ``out``: where dx goes (may be dsum itself)."""
    if stream is not None:
        return mx._under(stream, add_norm_backward, locals())
    torch = mx._torch()
    R, C = sum.shape
    dev = sum.device
    assert dy.dtype == torch.bfloat16 and dy.shape == sum.shape, "dy: BF16, of sum's shape"
    assert rstd.is_cuda and rstd.dtype == torch.float32 and rstd.is_contiguous() and rstd.numel() == R, "rstd: FP32, one per row"
    sd, ldd = mx._dtype(sum), 0
    if dsum is not None:
        assert dsum.dtype == sum.dtype and dsum.shape == sum.shape, "dsum: sum's dtype and shape"
        ldd = mx._rows(dsum)
    if out is None:
        out = torch.empty((R, C), dtype=sum.dtype, device=dev)
    assert out.dtype == sum.dtype and out.shape == sum.shape, "out: sum's dtype and shape"
    row, col, pointers, _, _ = _copies(axis, R, C, dev)
    dweight, ws, nbytes = None, None, 0
    if weight_grad:
        dweight = torch.empty(C, dtype=torch.float32, device=dev)
        nbytes = mx.mx_add_norm_backward_workspace_bytes(R, C)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    mx.mx_add_norm_backward(dy.data_ptr(), mx._rows(dy), sum.data_ptr(), mx._rows(sum), mx._ptr(dsum), ldd, sd, mx._ptr(weight),
                         mx._params(weight, None, C), rstd.data_ptr(), R, C, axis, out.data_ptr(), mx._rows(out), mx._ptr(dweight),
                         *pointers, mx._ptr(ws) if nbytes else None, nbytes, mx._ptr(status), mx._stream(stream))
    return AddNormGrads(out, dweight, row, col)


def gemm_gated(a: mx.MXTensor, gate: mx.MXTensor, up: mx.MXTensor, act: str = "silu", keep_preact: bool = False, out=None,
               status=None, stream=None):
    """act(A . gate^T) * (A . up^T) in BF16 [M, F] from row copies of the tokens
    and of the two weights. Returns (out, gate_up): with keep_preact the two
    products side by side, BF16 [M, 2F], for gated_backward_quantize, else None."""
    if stream is not None:
        return mx._under(stream, gemm_gated, locals())
    torch = mx._torch()
    M, F = a.rows, gate.rows
    dev = a.data.device
    if out is None:
        out = torch.empty((M, F), dtype=torch.bfloat16, device=dev)
    assert out.dtype == torch.bfloat16 and out.shape == (M, F), "out: BF16 [M, F]"
    pre = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=dev) if keep_preact else None
    mx.mx_gemm_gated(a.c_operand(), gate.c_operand(), up.c_operand(), mx.ACTIVATIONS[act], out.data_ptr(), mx._rows(out), mx._ptr(pre),
                  2 * F, mx._ptr(status), mx._stream(stream))
    return out, pre


def gated_quantize(gate_up, act: str = "silu", axis: int = mx.MX_BOTH, group_offsets=None, col_capacity: Optional[int] = None,
                   status=None, stream=None):
    """MX copies (row, col) of h = act(gate) * up from gate_up = [gate | up], BF16
    [rows, 2F]: what the down projection reads. ``group_offsets``, ``col_capacity``:
    the column copy in the experts' segments, as quantize's."""
    if stream is not None:
        return mx._under(stream, gated_quantize, locals())
    R, F = gate_up.shape[0], gate_up.shape[1] // 2
    assert gate_up.dtype == mx._torch().bfloat16 and gate_up.shape[1] % 2 == 0, "gate_up: BF16 [rows, 2F]"
    ld = mx._rows(gate_up)
    row, col, pointers, n_groups, cap = _copies(axis, R, F, gate_up.device, group_offsets, col_capacity)
    mx.mx_gated_quantize(gate_up.data_ptr(), ld, R, F, mx.ACTIVATIONS[act], axis, *pointers, mx._ptr(group_offsets), n_groups, cap,
                      mx._ptr(status), mx._stream(stream))
    return row, col


def gated_backward_quantize(dh, gate_up, act: str = "silu", axis: int = mx.MX_BOTH, group_offsets=None,
                            col_capacity: Optional[int] = None, status=None, stream=None):
    """MX copies (row, col) of [dgate | dup], [rows, 2F], from dh (BF16 [rows, F],
    the down projection's dgrad) and gate_up (BF16 [rows, 2F], gemm_gated's or
    grouped_gemm's): the dY of the two projections' dgrad and wgrad."""
    if stream is not None:
        return mx._under(stream, gated_backward_quantize, locals())
    R, F = dh.shape
    bf16 = mx._torch().bfloat16
    assert dh.dtype == bf16 and gate_up.dtype == bf16 and tuple(gate_up.shape) == (R, 2 * F), "dh BF16 [rows, F], gate_up [rows, 2F]"
    lddh, ld = mx._rows(dh), mx._rows(gate_up)
    row, col, pointers, n_groups, cap = _copies(axis, R, 2 * F, dh.device, group_offsets, col_capacity)
    mx.mx_gated_backward_quantize(dh.data_ptr(), lddh, gate_up.data_ptr(), ld, R, F, mx.ACTIVATIONS[act], axis, *pointers,
                               mx._ptr(group_offsets), n_groups, cap, mx._ptr(status), mx._stream(stream))
    return row, col
