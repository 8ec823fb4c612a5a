"""The gated block's calls through the C ABI with pitched matrices, in place and apart, and
guard bytes behind every buffer: nothing but the outputs is written, and those have
the bits of the packed call, which the oracle checks."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
from tests import test_gpu_add_norm as norm
from tests import test_gpu_gated as gate

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
GUARD = 512


def stream():
    return torch.cuda.current_stream().cuda_stream


class Copies:
    """Buffers for both copies of a [rows, cols] matrix, 0xA5 in them and behind them."""

    def __init__(self, rows, cols, axis, width=None):
        self.axis, sizes = axis, [rows * cols, mx.mx_scale_bytes(rows, cols), cols * (width or rows), mx.mx_scale_bytes(cols, width or rows)]
        self.sizes = [s if axis & (mx.MX_ROWWISE if i < 2 else mx.MX_COLWISE) else 0 for i, s in enumerate(sizes)]
        self.bufs = [torch.full((s + GUARD,), 0xA5, dtype=torch.uint8, device="cuda") for s in self.sizes]
        self.pointers = [b.data_ptr() if s else None for b, s in zip(self.bufs, self.sizes)]

    def check(self, row, col):
        torch.cuda.synchronize()
        want = [t for c in (row, col) for t in ((c.data, c.scale) if c is not None else (None, None))]
        for b, s, w in zip(self.bufs, self.sizes, want):
            assert (b[s:] == 0xA5).all()
            if s:
                assert torch.equal(b[:s], w.reshape(-1))


class Pitched:
    """A [rows, cols] output whose pitch gap, and a row behind it, hold 7."""

    def __init__(self, rows, cols, pad, dtype, like=None):
        self.buf = torch.full((rows + 1, cols + pad), 7.0, dtype=dtype, device="cuda")
        self.rows, self.cols = rows, cols
        self.m = self.buf[:rows, :cols]
        if like is not None:
            self.m.copy_(like)

    def arguments(self):
        return self.buf.data_ptr(), self.buf.stride(0)

    def check(self, want):
        torch.cuda.synchronize()
        assert torch.equal(self.m, want)
        assert (self.buf[:self.rows, self.cols:] == 7).all() and (self.buf[self.rows] == 7).all()


def vector(n):
    return torch.full((n + GUARD // 4,), -3.0, device="cuda")


# (rows, cols, stream, pad of its matrices, axis): partial warps, clusters, and dsum read by the lanes (FP32 above 8192 columns)
CASES = [(96, 608, BF16, 16, mx.MX_BOTH), (64, 1408, F32, 4, mx.MX_BOTH), (33, 96, BF16, 8, mx.MX_ROWWISE), (1, 2048, BF16, 24, mx.MX_ROWWISE),
         (160, 2048, BF16, 8, mx.MX_BOTH), (96, 7168, F32, 12, mx.MX_COLWISE), (32, 8224, F32, 8, mx.MX_BOTH), (64, 16384, F32, 4, mx.MX_BOTH),
         (64, 16384, BF16, 8, mx.MX_BOTH), (40, 352, F32, 4, 0), (7072, 544, BF16, 8, mx.MX_BOTH)]


@pytest.mark.parametrize("rows,cols,dtype,pad,axis", CASES)
def test_norm_forward(rows, cols, dtype, pad, axis):
    x, res, w = norm.matrix(rows, cols, 1, BF16, 8), norm.matrix(rows, cols, 2, dtype, pad), norm.weight_of(cols, 3)
    want = mx.add_norm_quantize(x, res, w, eps=norm.EPS, axis=axis, keep_output=True)
    norm.check_forward(want, x, res, w)
    code = mx.MX_F32 if dtype == F32 else mx.MX_BF16
    for apart in (True, False):
        total = Pitched(rows, cols, pad + (16 if apart else 0), dtype, None if apart else res)
        y, rstd, copies = Pitched(rows, cols, 32, BF16), vector(rows), Copies(rows, cols, axis)
        stream_in = (res.data_ptr(), cols + pad) if apart else total.arguments()
        mx.mx_add_norm_quantize(x.data_ptr(), cols + 8, *stream_in, code, w.data_ptr(), mx.MX_F32, rows, cols, norm.EPS, axis,
                                *total.arguments(), *y.arguments(), rstd.data_ptr(), *copies.pointers, None, stream())
        total.check(want.sum)
        y.check(want.y)
        copies.check(want.row, want.col)
        assert torch.equal(rstd[:rows], want.rstd) and (rstd[rows:] == -3).all()


@pytest.mark.parametrize("with_dsum", [True, False])
@pytest.mark.parametrize("rows,cols,dtype,pad,axis", CASES)
def test_norm_backward(rows, cols, dtype, pad, axis, with_dsum):
    """dx apart, over dsum, and not wanted where there are copies."""
    s, dy = norm.matrix(rows, cols, 4, dtype, pad, std=2.0), norm.matrix(rows, cols, 5, BF16, 8, std=0.1)
    ds = norm.matrix(rows, cols, 6, dtype, pad, std=0.3) if with_dsum else None
    w = norm.weight_of(cols, 7)
    rstd = torch.from_numpy(norm.so.norm_stats(norm.f64(s), norm.EPS, False)[1].astype(np.float32)).cuda()
    want = mx.add_norm_backward(dy, s, w, rstd, dsum=ds, axis=axis)
    norm.check_backward(want, dy, s, w, rstd, ds)
    code = mx.MX_F32 if dtype == F32 else mx.MX_BF16
    need = mx.mx_add_norm_backward_workspace_bytes(rows, cols)
    for how in ("apart", "in place", "none"):
        if (how == "in place" and not with_dsum) or (how == "none" and axis == 0):
            continue
        dx = Pitched(rows, cols, pad + (16 if how == "apart" else 0), dtype, ds if how == "in place" else None)
        dsum = dx.arguments() if how == "in place" else (ds.data_ptr(), cols + pad) if with_dsum else (None, 0)
        dw, copies = vector(cols), Copies(rows, cols, axis)
        ws = torch.full((need + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        mx.mx_add_norm_backward(dy.data_ptr(), cols + 8, s.data_ptr(), cols + pad, *dsum, code, w.data_ptr(), mx.MX_F32,
                                rstd.data_ptr(), rows, cols, axis, *(dx.arguments() if how != "none" else (None, 0)), dw.data_ptr(),
                                *copies.pointers, ws.data_ptr(), need, None, stream())
        copies.check(want.row, want.col)
        if how == "none":
            assert (dx.buf == 7).all()
        else:
            dx.check(want.dx)
        assert torch.equal(dw[:cols], want.dweight) and (dw[cols:] == -3).all() and (ws[need:] == 0xA5).all()


# last tiles of 32, 64, 96 rows, last units of 32 columns
@pytest.mark.parametrize("axis", [mx.MX_ROWWISE, mx.MX_COLWISE, mx.MX_BOTH])
@pytest.mark.parametrize("rows", [32, 64, 96, 160, 192, 224])
@pytest.mark.parametrize("F", [32, 96, 160, 352])
def test_gate_dense(rows, F, axis):
    check_gate(rows, F, axis, {})


@pytest.mark.parametrize("rows,F", [(1, 32), (31, 96), (129, 160), (300, 1408)])
def test_gate_row_copies(rows, F):
    check_gate(rows, F, mx.MX_ROWWISE, {})


@pytest.mark.parametrize("axis", [mx.MX_COLWISE, mx.MX_BOTH])
@pytest.mark.parametrize("counts,F", [([100, 0, 156], 96), ([37, 0, 300, 1, 128], 352), ([0, 0, 129], 32), ([256], 1408), ([0] * 511 + [33], 64)])
def test_gate_groups(counts, F, axis):
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    check_gate(int(offs[-1]), F, axis, dict(group_offsets=torch.from_numpy(offs).cuda(), col_capacity=mx.mx_grouped_padded_rows(offs)), offs)


def check_gate(rows, F, axis, groups, offs=None):
    z, dh = gate.normal(rows, 2 * F, 21, 2.0, 8), gate.normal(rows, F, 22, 0.1, 16)
    h, b = mx.gated_quantize(z, axis=axis, **groups), mx.gated_backward_quantize(dh, z, axis=axis, **groups)
    gate.check_gate(z, dh, "silu", *h, *b, offsets=offs)
    cap = groups.get("col_capacity", 0)
    tail = (groups["group_offsets"].data_ptr(), len(offs) - 1, cap) if groups else (None, 0, 0)
    copies = Copies(rows, F, axis, cap)
    mx.mx_gated_quantize(z.data_ptr(), 2 * F + 8, rows, F, mx.MX_ACT_SILU, axis, *copies.pointers, *tail, None, stream())
    copies.check(*h)
    copies = Copies(rows, 2 * F, axis, cap)
    mx.mx_gated_backward_quantize(dh.data_ptr(), F + 16, z.data_ptr(), 2 * F + 8, rows, F, mx.MX_ACT_SILU, axis, *copies.pointers, *tail,
                                  None, stream())
    copies.check(*b)
