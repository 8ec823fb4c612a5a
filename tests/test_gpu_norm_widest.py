"""Rows near the largest width a norm accepts (2**31 - 1 columns), where a column's
index, a step past it and the second half of a partial row pass 31 bits.

The entries are small whole numbers and the statistics handed to the backward pass
are 0 and 1, so its sums (per thread below 2**24) are exact but for the last ten
additions, and dweight and dbias are exact. The forward pass's variance is a chain
of 2**21 additions per thread: off by 2**21 * 2**-24 = 1/8 at most, its root by 1/16.
"""
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx

pytestmark = pytest.mark.gpu
PIECE = 1 << 26


def pieces(cols):
    return [(c, min(c + PIECE, cols)) for c in range(0, cols, PIECE)]


def whole(row, a, b, salt):
    """Entries -2, -1, 1, 2 of columns a .. b, by a hash of row and column."""
    c = torch.arange(a, b, device="cuda", dtype=torch.int64) + (salt + 7 * row) * 1000003
    h = ((c * 0x9E3779B1) >> 13) & 3
    return torch.tensor([-2.0, -1.0, 1.0, 2.0], device="cuda")[h]


def matrix(rows, cols, salt):
    t = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    for r in range(rows):
        for a, b in pieces(cols):
            t[r, a:b] = whole(r, a, b, salt)
    return t


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


# 2**30 + 8: the second half of a partial row; 2**31 - 8: 16-byte vectors; 2**31 - 1: single elements
@pytest.mark.parametrize("rows,cols", [(2, 2 ** 30 + 8), (1, 2 ** 31 - 8), (1, 2 ** 31 - 1)])
def test_backward(rows, cols):
    x, dy = matrix(rows, cols, 1), matrix(rows, cols, 2)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    s1, s2 = [0] * rows, [0] * rows
    for r in range(rows):
        for a, b in pieces(cols):
            p, q = x[r, a:b].float(), dy[r, a:b].float()
            s1[r] += int(q.double().sum())
            s2[r] += int((p * q).double().sum())
    st = mx.new_status()
    dx, dw, db = mx.layer_norm_backward(dy, x, None, mean, rstd, status=st)
    assert mx.read_status(st) == 0
    for a, b in pieces(cols):
        p, q = x[:, a:b].float(), dy[:, a:b].float()
        assert torch.equal(dw[a:b], (p * q).sum(0)) and torch.equal(db[a:b], q.sum(0)), (a, b)
        for r in range(rows):
            want = q[r] - s1[r] / cols - p[r] * (s2[r] / cols)
            assert ((dx[r, a:b].float() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all(), (r, a, b)


@pytest.mark.parametrize("rows,cols", [(1, 2 ** 31 - 8), (1, 2 ** 31 - 1)])
def test_forward(rows, cols):
    x = matrix(rows, cols, 3)
    sq = sum(float(x[0, a:b].float().square().double().sum()) for a, b in pieces(cols))
    y, mean, rstd = mx.layer_norm(x, eps=0.0)
    want = (sq / cols) ** -0.5
    assert abs(float(mean)) < 1e-3 and abs(float(rstd) / want - 1) < 0.07
    for a, b in pieces(cols):
        ref = x[0, a:b].float() * want
        assert ((y[0, a:b].float() - ref).abs() <= (0.07 + 2.0 ** -8) * ref.abs() + 2e-3).all(), (a, b)
