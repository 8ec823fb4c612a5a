"""The gated block's calls on tensors past 2^31 elements: sampled rows and columns, the
last ones among them. Inputs are drawn on the device (seeded)."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import oracle
from oracle import step_oracle as so
from tests import test_gpu_add_norm as norm
from tests import test_gpu_gated as gate
from tests.gpu_util import f64, u8
from tests.test_gpu_large import device_normal

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def scales_of(copy, rows, blocks):
    """Logical scales [len(rows), len(blocks)] of a copy whose buffer is too large to unfold whole."""
    r, b = np.asarray(rows)[:, None], np.asarray(blocks)[None]
    ka = -(-copy.k // 128)
    at = ((r >> 7) * ka + (b >> 2)) * 512 + ((r & 31) << 4) + (((r >> 5) & 3) << 2) + (b & 3)
    return u8(copy.scale[torch.from_numpy(at.reshape(-1)).cuda()]).reshape(at.shape)


def check_rows(copy, rows, ref, tol, what):
    codes = u8(copy.data[torch.as_tensor(rows, device="cuda")])
    assert so.copy_error(codes, scales_of(copy, rows, np.arange(copy.k // 32)), ref, tol) <= 0, what


def check_panel(copy, cols, row0, ref, tol, what):
    """Of a column copy: columns `cols` of the 32 rows from row0 on; ref [32, len(cols)]."""
    codes = u8(copy.data[torch.as_tensor(cols, device="cuda")][:, row0:row0 + 32])
    assert so.copy_error(codes, scales_of(copy, cols, [row0 // 32]), ref.T, tol.T) <= 0, what


def test_norm():
    R, C = 131104, 16384                      # 2.148e9 elements
    assert R * C > 2 ** 31
    x, res, w = device_normal((R, C), 1, 0.5), device_normal((R, C), 2, 2.0), norm.weight_of(C, 3)
    st = mx.new_status()
    n = mx.add_norm_quantize(x, res, w, eps=norm.EPS, status=st)
    assert mx.read_status(st) == 0
    rows = [0, 1, 31, 65535, 65536, R - 33] + list(range(R - 32, R))
    at = torch.tensor(rows, device="cuda")
    v, rstd, y = so.add_norm(f64(x[at]), f64(res[at]), norm.f64(w), norm.EPS)
    norm.check(n.sum[at], v, (norm.U + norm.ROUND[BF16]) * np.abs(v), "sum")
    norm.check(n.rstd[at], rstd, 36 * norm.U * rstd, "rstd")
    tol = 40 * norm.U * np.abs(y)
    check_rows(n.row, rows, y, tol, "row copy")
    cols = [0, 1, 31, 8000, C - 1]
    check_panel(n.col, cols, R - 32, y[-32:, cols], tol[-32:, cols], "column copy")
    del x, n.row, n.col

    dy, s = device_normal((R, C), 4, 0.1), n.sum
    b = mx.add_norm_backward(dy, s, w, n.rstd, dsum=res, axis=mx.MX_BOTH, status=st)
    assert mx.read_status(st) == 0
    fy, fs, fr, fd = f64(dy[at]), f64(s[at]), norm.f64(n.rstd[at]), f64(res[at])
    dx, _ = so.add_norm_backward(fy, fs, norm.f64(w), fr, fd)
    tol = norm.backward_tolerance(fy, fs, norm.f64(w), fr, fd)
    norm.check(b.dx[at], dx, tol + norm.ROUND[BF16] * (np.abs(dx) + tol), "dx")
    check_rows(b.row, rows, dx, tol, "dx row copy")
    check_panel(b.col, cols, R - 32, dx[-32:, cols], tol[-32:, cols], "dx column copy")
    # a column's sum over all rows, in 64 bits. A lane adds 8 rows of a panel, 4 lanes their sums, a cluster its
    # panels' (there are 4 clusters of 16 CTAs at least), 32 threads the clusters': a chain of at most
    terms = dy[:, cols].double() * s[:, cols].double() * n.rstd.double()[:, None]
    chain = 8 + 2 + -(-(R // 32) // 4) + 32 + 3       # and each term's three roundings
    assert ((b.dweight[cols].double() - terms.sum(0)).abs() <= chain * norm.U * terms.abs().sum(0)).all()


@pytest.mark.parametrize("groups", [False, True])
def test_gate(groups):
    R, F = 98336, 11008                       # [gate | up] and its gradient: 2.165e9 elements
    assert R * 2 * F > 2 ** 31
    z, dh = device_normal((R, 2 * F), 5), device_normal((R, F), 6, 0.1)
    offs = np.array([0, 40000, 40000, 40001, R])
    kw = dict(group_offsets=torch.from_numpy(offs).cuda(), col_capacity=mx.mx_grouped_padded_rows(offs)) if groups else {}
    st = mx.new_status()
    row, col = mx.gated_quantize(z, status=st, **kw)
    brow, bcol = mx.gated_backward_quantize(dh, z, status=st, **kw)
    assert mx.read_status(st) == 0
    rows = [0, 1, 48770, 48771, R - 33] + list(range(R - 32, R))
    at = torch.tensor(rows, device="cuda")
    zz, d = f64(z[at]), f64(dh[at])
    g, u = zz[:, :F], zz[:, F:]
    th, tg, tu = gate.gate_tolerances(d, g, u, "silu")
    h, dz, tz = so.gated(g, u, "silu"), np.concatenate(so.gated_backward(d, g, u, "silu"), 1), np.concatenate([tg, tu], 1)
    check_rows(row, rows, h, th, "h")
    check_rows(brow, rows, dz, tz, "dgate dup")
    # the last whole block of 32 rows of the column copies: of the last group, from row 40001 on
    start, first = (40001, sum(-(-n // 128) * 128 for n in (40000, 0, 1))) if groups else (0, 0)
    block = (R - start) // 32 - 1
    lo = start + 32 * block
    zz, d = f64(z[lo:lo + 32]), f64(dh[lo:lo + 32])
    g, u = zz[:, :F], zz[:, F:]
    th, tg, tu = gate.gate_tolerances(d, g, u, "silu")
    h, dz, tz = so.gated(g, u, "silu"), np.concatenate(so.gated_backward(d, g, u, "silu"), 1), np.concatenate([tg, tu], 1)
    for copy, ref, tol in ((col, h, th), (bcol, dz, tz)):
        cols = [0, 31, 5000, ref.shape[1] - 1]
        check_panel(copy, cols, first + 32 * block, ref[:, cols], tol[:, cols], "columns")


@pytest.mark.parametrize("M,F", [(98336, 11008), (98304, 11001), (17, 1 << 26)])
def test_product(M, F):
    """Both projections kept: whole tiles with aligned rows and without, and few tokens."""
    K = 32
    assert M * 2 * F > 2 ** 31
    a, gt, up = device_normal((M, K), 7), device_normal((F, K), 8, 0.3), device_normal((F, K), 9, 0.3)
    st = mx.new_status()
    qa, qg, qu = (mx.quantize(t, mx.MX_ROWWISE, status=st)[0] for t in (a, gt, up))
    out, pre = mx.gemm_gated(qa, qg, qu, keep_preact=True, status=st)
    assert mx.read_status(st) == 0
    rows = sorted({0, 1, M // 2, M - 2, M - 1})
    cols = sorted({0, 1, 127, 128, F // 2, F - 2, F - 1})
    qr, qc = torch.tensor(rows, device="cuda"), torch.tensor(cols, device="cuda")
    ca, sa = oracle.mx_quantize_rowwise(f64(a[qr]))
    (g, sg), (u, su) = (oracle.mx_gemm_ref(ca, sa, *oracle.mx_quantize_rowwise(f64(t[qc]))) for t in (gt, up))
    got = f64(out[qr][:, qc]), f64(pre[qr][:, qc]), f64(pre[qr][:, qc + F])
    ref = so.gated(g, u, "silu")
    tol = 1.13 * 1e-6 * sg * (np.abs(u) + 1e-6 * su) + np.abs(so.act(g, "silu")) * 1e-6 * su + 2.0 ** -14 * np.abs(ref)
    assert (np.abs(got[0] - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol)).all()
    for z, r, s in ((got[1], g, sg), (got[2], u, su)):
        assert (np.abs(z - r) <= 1e-6 * s + 2.0 ** -8 * (np.abs(r) + 1e-6 * s)).all()
