"""MX copies of computed values against the float64 oracle."""
import numpy as np

import oracle
from oracle import step_oracle as so
from tests.gpu_util import u8


def logical(copy):
    """(codes, scales) of an MXTensor; the buffer's padding has to be zero."""
    scales = oracle.mx_scale_unswizzle(u8(copy.scale), copy.rows, copy.k // 32)
    assert np.array_equal(oracle.mx_scale_swizzle(scales), u8(copy.scale)), "scale padding"
    return u8(copy.data), scales


def check_copy(copy, ref, tol, what):
    """The copy of [rows, k] values that are within tol of ref."""
    assert (copy.rows, copy.k) == ref.shape, (what, copy.rows, copy.k, ref.shape)
    codes, scales = logical(copy)
    off = so.copy_error(codes, scales, ref, tol)
    assert off <= 0, (what, off)


def check_copies(row, col, ref, tol, what, offsets=None):
    tol = np.broadcast_to(tol, ref.shape)
    if row is not None:
        check_copy(row, ref, tol, what + " row copy")
    if col is not None:
        if offsets is not None:
            ref, tol = so.segments(ref, offsets), so.segments(tol, offsets)
        check_copy(col, ref.T, tol.T, what + " column copy")


def check_exact(row, col, values, what, offsets=None):
    """Byte for byte the quantiser's oracle on these values."""
    if row is not None:
        d, s = oracle.mx_quantize_rowwise(values)
        assert np.array_equal(u8(row.data), d), (what, "row codes", np.argwhere(u8(row.data) != d)[:4].tolist())
        assert np.array_equal(u8(row.scale), oracle.mx_scale_swizzle(s)), (what, "row scales")
    if col is not None:
        if offsets is None:
            d, s = oracle.mx_quantize_colwise(values)
        else:
            d, s = oracle.mx_quantize_colwise_grouped(values, offsets)[:2]
        assert np.array_equal(u8(col.data), d), (what, "column codes", np.argwhere(u8(col.data) != d)[:4].tolist())
        assert np.array_equal(u8(col.scale), oracle.mx_scale_swizzle(s)), (what, "column scales")
