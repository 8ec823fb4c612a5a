"""The residual's addition, the root-mean-square norm and its MX copies, and the
backward pass, against the float64 oracle.

Tolerances (u = 2**-24). v = x + residual is one rounding. A row's sum of squares is
a chain of at most 60 additions (8 pairs of a lane, 3 in a warp, 16 warps, 16 CTAs,
and what a pairwise step adds), so the variance is off by 64u of itself (v's own
rounding twice among them), 1/sqrt by half of that and 4 roundings: 36u; y by two
products more and v's rounding: 40u. Backward, the row's mean of g h the same way:
off by 64u of the mean of magnitudes (h and g are one rounding each); dx adds at
most six roundings of each of its three terms. A sum over rows is a chain of at most
200 additions here. BF16 rounds by 2**-8 of the value at most.
"""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import oracle
import workloads
from oracle import step_oracle as so
from tests.copies import check_copies, check_exact, logical

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ROUND = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def f64(t):
    return t.detach().double().cpu().numpy()


def matrix(rows, cols, seed, dtype, pad=0, std=1.0, fill=float("nan")):
    """Normal values, a hundredth of the columns 20 times as large, in a buffer whose pitch gap holds `fill`."""
    r = workloads.philox(seed)
    a = r.standard_normal((rows, cols)) * std * np.where(r.random(cols) < 0.01, 20.0, 1.0)
    buf = torch.full((rows, cols + pad), fill, dtype=dtype, device="cuda")
    t = buf[:, :cols]
    t.copy_(torch.from_numpy(a.astype(np.float32)))
    return t


def weight_of(cols, seed, dtype=F32):
    return (1.0 + 0.2 * torch.from_numpy(workloads.philox(seed).standard_normal(cols).astype(np.float32))).cuda().to(dtype)


def check(got, ref, tol, what):
    got = f64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], ref[bad][:3])


def check_forward(n, x, residual, weight, eps=EPS):
    fx, fr = f64(x), 0.0 if residual is None else f64(residual)
    fw = np.ones(fx.shape[1]) if weight is None else f64(weight)
    v, rstd, y = so.add_norm(fx, fr, fw, eps)
    if residual is not None:
        check(n.sum, v, U * np.abs(v) + ROUND[n.sum.dtype] * np.abs(v), "sum")
    check(n.rstd, rstd, 36 * U * rstd, "rstd")
    tol = 40 * U * np.abs(y)
    if n.y is not None:
        check(n.y, y, tol + ROUND[BF16] * (np.abs(y) + tol), "y")
    check_copies(n.row, n.col, y, tol, "y")


def backward_tolerance(dy, v, w, rstd, ds):
    h, g, r = v * rstd[:, None], dy * w, rstd[:, None]
    m = (g * h).mean(1, keepdims=True)
    return 6 * U * (r * np.abs(g) + np.abs(ds) + np.abs(h * r * m)) + 64 * U * np.abs(h) * r * np.abs(g * h).mean(1, keepdims=True)


def check_backward(b, dy, s, weight, rstd, dsum):
    fy, fs, fr = f64(dy), f64(s), f64(rstd)
    fw = np.ones(fs.shape[1]) if weight is None else f64(weight)
    fd = np.zeros_like(fs) if dsum is None else f64(dsum)
    dx, dw = so.add_norm_backward(fy, fs, fw, fr, fd)
    tol = backward_tolerance(fy, fs, fw, fr, fd)
    check(b.dx, dx, tol + ROUND[b.dx.dtype] * (np.abs(dx) + tol), "dx")
    if b.dweight is not None:
        check(b.dweight, dw, 200 * U * np.abs(fy * fs * fr[:, None]).sum(0), "dweight")
    check_copies(b.row, b.col, dx, tol, "dx")


# columns around every way a row is split: part of a warp's 64, several warps, clusters of 2 to 16, sixteen warps a CTA
WIDTHS = [32, 64, 96, 160, 512, 544, 1408, 2048, 4128, 7168, 8192, 8224, 10272, 16384]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", WIDTHS)
def test_forward_widths(cols, dtype):
    rows = 64 if cols > 4096 else 160
    x, res, w = matrix(rows, cols, 1, BF16, std=0.5), matrix(rows, cols, 2, dtype, std=2.0), weight_of(cols, 3)
    st = mx.new_status()
    n = mx.add_norm_quantize(x, res, w, eps=EPS, axis=mx.MX_BOTH, keep_output=True, status=st)
    assert mx.read_status(st) == 0
    check_forward(n, x, res, w)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", WIDTHS)
def test_backward_widths(cols, dtype):
    rows = 64 if cols > 4096 else 160
    s, dy, ds = matrix(rows, cols, 4, dtype, std=2.0), matrix(rows, cols, 5, BF16, std=0.1), matrix(rows, cols, 6, dtype, std=0.3)
    w = weight_of(cols, 7)
    rstd = torch.from_numpy(so.norm_stats(f64(s), EPS, False)[1].astype(np.float32)).cuda()
    st = mx.new_status()
    b = mx.add_norm_backward(dy, s, w, rstd, dsum=ds, axis=mx.MX_BOTH, status=st)
    assert mx.read_status(st) == 0
    check_backward(b, dy, s, w, rstd, ds)


# panels enough for several rounds of every cluster, two CTAs an SM
@pytest.mark.parametrize("rows,cols,dtype", [(5152, 2048, BF16), (2080, 7168, BF16), (2592, 4096, BF16), (4224, 1024, F32), (1056, 7168, F32),
                                             (1312, 5120, BF16), (1312, 5120, F32), (992, 6144, F32)])
def test_rounds(rows, cols, dtype):
    x, res, w = matrix(rows, cols, 1, BF16, std=0.5), matrix(rows, cols, 2, dtype, std=2.0), weight_of(cols, 3)
    n = mx.add_norm_quantize(x, res, w, eps=EPS, axis=mx.MX_BOTH, keep_output=True)
    check_forward(n, x, res, w)
    dy, ds = matrix(rows, cols, 5, BF16, std=0.1), matrix(rows, cols, 6, dtype, std=0.3)
    for axis, dsum in ((mx.MX_BOTH, ds), (mx.MX_ROWWISE, None), (0, ds)):
        check_backward(mx.add_norm_backward(dy, n.sum, w, n.rstd, dsum=dsum, axis=axis), dy, n.sum, w, n.rstd, dsum)


@pytest.mark.parametrize("rows", [1, 2, 31, 32, 33, 127, 129, 1000])
@pytest.mark.parametrize("cols,pad,dtype", [(96, 8, BF16), (2048, 64, BF16), (1408, 4, F32)])
def test_row_counts(rows, cols, pad, dtype):
    """Row copies (and none) of any number of rows, with row pitches."""
    xpad = 8 * (pad // 4)
    x, res, w = matrix(rows, cols, 11, BF16, xpad), matrix(rows, cols, 12, dtype, pad), weight_of(cols, 13, BF16)
    n = mx.add_norm_quantize(x, res, w, eps=EPS, axis=mx.MX_ROWWISE)
    assert n.col is None and n.y is None
    check_forward(n, x, res, w)
    n = mx.add_norm_quantize(x, res, w, eps=EPS, axis=0, keep_output=True)
    check_forward(n, x, res, w)
    dy, ds = matrix(rows, cols, 14, BF16, xpad, std=0.1), matrix(rows, cols, 15, dtype, pad)
    for axis in (0, mx.MX_ROWWISE):
        check_backward(mx.add_norm_backward(dy, n.sum, w, n.rstd, dsum=ds, axis=axis), dy, n.sum, w, n.rstd, ds)


@pytest.mark.parametrize("axis", [mx.MX_ROWWISE, mx.MX_COLWISE, mx.MX_BOTH])
def test_without_residual_weight_or_gradient(axis):
    x = matrix(96, 352, 21, BF16)
    n = mx.add_norm_quantize(x, eps=EPS, axis=axis)
    assert n.sum is x
    check_forward(n, x, None, None)
    dy = matrix(96, 352, 22, BF16)
    b = mx.add_norm_backward(dy, n.sum, None, n.rstd, axis=axis)
    check_backward(b, dy, x, None, n.rstd, None)
    b = mx.add_norm_backward(dy, n.sum, None, n.rstd, axis=axis, weight_grad=False)
    assert b.dweight is None
    check_backward(b, dy, x, None, n.rstd, None)


def test_codes_bit_for_bit():
    """Rows of one magnitude, +-2^k, and eps 0: rstd is 2^-k and y = +-weight exactly,
    so the copies are the quantiser's of the FP32 weight, byte for byte."""
    rows, cols = 96, 416
    r = workloads.philox(31)
    sign = np.where(r.random((rows, cols)) < 0.5, -1.0, 1.0)
    k = np.exp2(r.integers(-30, 30, (rows, 1)).astype(np.float64))
    w = (r.standard_normal(cols) * np.exp2(r.integers(-60, 60, cols).astype(np.float64))).astype(np.float32)
    w[64:96] = 0.0
    w[100] = 448.0
    w[130] = 2.0 ** -140                    # subnormal
    x = torch.from_numpy((sign * k).astype(np.float32)).cuda().to(BF16)
    n = mx.add_norm_quantize(x, None, torch.from_numpy(w).cuda(), eps=0.0, keep_output=True)
    assert np.array_equal(f64(n.rstd), 1 / k[:, 0])
    check_exact(n.row, n.col, sign * w.astype(np.float64), "y")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_values(bad):
    """A row with NaN (or an infinity, whose norm is NaN at its place) spoils its own
    blocks and the columns' that cross it; the other rows' row blocks are right."""
    rows, cols = 64, 192
    x, res, w = matrix(rows, cols, 41, BF16), matrix(rows, cols, 42, BF16), weight_of(cols, 43)
    x[40, 70] = bad
    n = mx.add_norm_quantize(x, res, w, eps=EPS, keep_output=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        _, _, y = so.add_norm(f64(x), f64(res), f64(w), EPS)
    y[40, :] = np.nan if np.isnan(bad) else 0.0
    y[40, 70] = np.nan
    got = f64(n.y)
    assert np.array_equal(np.isnan(got), np.isnan(y))
    codes, scales = logical(n.row)
    _, want = oracle.mx_quantize_rowwise(y)
    assert np.array_equal(scales == 0xFF, want == 0xFF)
    assert ((codes[40, 64:96] & 0x7F) == 0x7F).all()
    keep = [i for i in range(rows) if i != 40]
    assert so.copy_error(codes[keep], scales[keep], y[keep], 40 * U * np.abs(y[keep])) <= 0
    codes, scales = logical(n.col)
    _, want = oracle.mx_quantize_colwise(y)
    assert np.array_equal(scales == 0xFF, want == 0xFF)
    assert ((codes[70, 32:] & 0x7F) == 0x7F).all()


def test_zero_rows_and_zero_values():
    w = weight_of(64, 51)
    n = mx.add_norm_quantize(torch.zeros(0, 64, dtype=BF16, device="cuda"), None, w)
    assert n.row.data.numel() == 0
    b = mx.add_norm_backward(torch.zeros(0, 64, dtype=BF16, device="cuda"), n.sum, w, n.rstd)
    assert (b.dweight == 0).all() and b.dweight.shape == (64,)
    z = torch.zeros(32, 64, dtype=BF16, device="cuda")
    n = mx.add_norm_quantize(z, z, w, eps=EPS, keep_output=True)
    assert (n.y == 0).all()
    check_exact(n.row, n.col, np.zeros((32, 64)), "zeros")


def test_in_place():
    """The sum over the residual, dx over dsum."""
    for dtype in (BF16, F32):
        x, res, w = matrix(320, 1408, 61, BF16, 8), matrix(320, 1408, 62, dtype, 8), weight_of(1408, 63)
        a = mx.add_norm_quantize(x, res, w, eps=EPS)
        mine = res.clone()
        b = mx.add_norm_quantize(x, mine, w, eps=EPS, out=mine)
        assert b.sum is mine and torch.equal(a.sum, b.sum) and torch.equal(a.row.data, b.row.data) and torch.equal(a.col.data, b.col.data)
        dy, ds = matrix(320, 1408, 64, BF16), matrix(320, 1408, 65, dtype)
        g = mx.add_norm_backward(dy, a.sum, w, a.rstd, dsum=ds, axis=mx.MX_BOTH)
        mine = ds.clone()
        h = mx.add_norm_backward(dy, a.sum, w, a.rstd, dsum=mine, axis=mx.MX_BOTH, out=mine)
        assert torch.equal(g.dx, h.dx) and torch.equal(g.dweight, h.dweight) and torch.equal(g.col.data, h.col.data)


def test_untouched_neighbours_and_same_bits():
    """Pitch gaps and the bytes behind every buffer stay as they were; a second call gives the same bits."""
    rows, cols, pad = 96, 608, 16
    x, res, w = matrix(rows, cols, 71, BF16, pad), matrix(rows, cols, 72, BF16, pad), weight_of(cols, 73)
    gap = torch.full((rows + 1, cols + pad), 7.0, dtype=BF16, device="cuda")
    n1 = mx.add_norm_quantize(x, res, w, eps=EPS, out=gap[:rows, :cols])
    assert (gap[:rows, cols:] == 7).all() and (gap[rows] == 7).all()
    n2 = mx.add_norm_quantize(x, res, w, eps=EPS)
    for a, b in ((n1.sum, n2.sum), (n1.rstd, n2.rstd), (n1.row.data, n2.row.data), (n1.col.scale, n2.col.scale)):
        assert torch.equal(a, b)
    guard = 256
    sizes = [rows * cols, mx.mx_scale_bytes(rows, cols), rows * cols, mx.mx_scale_bytes(cols, rows)]
    bufs = [torch.full((s + guard,), 0xA5, dtype=torch.uint8, device="cuda") for s in sizes]
    rstd = torch.full((rows + 32,), -1.0, device="cuda")
    mx.mx_add_norm_quantize(x.data_ptr(), cols + pad, res.data_ptr(), cols + pad, mx.MX_BF16, w.data_ptr(), mx.MX_F32, rows, cols,
                            EPS, mx.MX_BOTH, None, 0, None, 0, rstd.data_ptr(), *[b.data_ptr() for b in bufs], None,
                            torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    for b, s in zip(bufs, sizes):
        assert (b[s:] == 0xA5).all()
    assert (rstd[rows:] == -1).all()
    assert torch.equal(bufs[0][:sizes[0]].view(rows, cols), n1.row.data) and torch.equal(bufs[3][:sizes[3]], n1.col.scale)


def test_many_panels_a_cluster():
    """More panels than clusters at once: every warp's ring goes round."""
    rows, cols = 32 * 700, 544
    x, res, w = matrix(rows, cols, 81, BF16), matrix(rows, cols, 82, BF16), weight_of(cols, 83)
    n = mx.add_norm_quantize(x, res, w, eps=EPS)
    check_forward(n, x, res, w)
    dy, ds = matrix(rows, cols, 84, BF16, std=0.1), matrix(rows, cols, 85, BF16)
    b = mx.add_norm_backward(dy, n.sum, w, n.rstd, dsum=ds, axis=mx.MX_BOTH)
    fy, fs, fr = f64(dy), f64(n.sum), f64(n.rstd)
    dx, dw = so.add_norm_backward(fy, fs, f64(w), fr, f64(ds))
    tol = backward_tolerance(fy, fs, f64(w), fr, f64(ds))
    check(b.dx, dx, tol + ROUND[BF16] * (np.abs(dx) + tol), "dx")
    check_copies(b.row, b.col, dx, tol, "dx")
    # 700 panels over at least 76 clusters: a lane's chain is at most 4 * 10 rows, the partial rows' 608 / 32 + 5
    check(b.dweight, dw, 200 * U * np.abs(fy * fs * fr[:, None]).sum(0), "dweight")


def test_gradients_against_differences():
    """The GPU's gradients against central differences of the float64 forward pass."""
    rows, cols = 32, 64
    x, res, w = matrix(rows, cols, 91, BF16), matrix(rows, cols, 92, F32), weight_of(cols, 93)
    dy, ds = matrix(rows, cols, 94, BF16), matrix(rows, cols, 95, F32)
    n = mx.add_norm_quantize(x, res, w, eps=0.1)
    b = mx.add_norm_backward(dy, n.sum, w, n.rstd, dsum=ds)
    fx, fr, fw, fy, fd = map(f64, (x, res, w, dy, ds))

    def loss(x_, w_):
        v, _, y = so.add_norm(x_, fr, w_, 0.1)
        return float((y * fy).sum() + (v * fd).sum())

    h = 1e-4
    for i, j in [(0, 0), (5, 17), (31, 63), (12, 40)]:
        e = np.zeros_like(fx)
        e[i, j] = h
        d = (loss(fx + e, fw) - loss(fx - e, fw)) / (2 * h)
        assert abs(d - float(b.dx[i, j])) <= 1e-5 * max(1.0, abs(d))
    for j in (0, 31, 63):
        e = np.zeros_like(fw)
        e[j] = h
        d = (loss(fx, fw + e) - loss(fx, fw - e)) / (2 * h)
        assert abs(d - float(b.dweight[j])) <= 1e-5 * max(1.0, abs(d))


def test_streams_and_graph():
    """On a stream of its own, and captured and replayed on new inputs."""
    rows, cols = 512, 2048
    x, res, w = matrix(rows, cols, 101, BF16), matrix(rows, cols, 102, BF16), weight_of(cols, 103)
    dy, ds = matrix(rows, cols, 104, BF16), matrix(rows, cols, 105, BF16)

    def step():
        n = mx.add_norm_quantize(x, res, w, eps=EPS)
        return n, mx.add_norm_backward(dy, n.sum, w, n.rstd, dsum=ds, axis=mx.MX_BOTH)

    def tensors(o):
        n, b = o
        return [n.sum, n.rstd, n.row.data, n.row.scale, n.col.data, n.col.scale, b.dx, b.dweight, b.row.data, b.col.data]

    want = [t.clone() for t in tensors(step())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = mx.add_norm_quantize(x, res, w, eps=EPS, stream=side)
    b = mx.add_norm_backward(dy, n.sum, w, n.rstd, dsum=ds, axis=mx.MX_BOTH, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(tensors((n, b)), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    x2 = matrix(rows, cols, 106, BF16)
    keep = x.clone()
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    new = [t.clone() for t in tensors(held)]
    assert all(torch.equal(p, q) for p, q in zip(tensors(step()), new))
    x.copy_(keep)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(tensors(held), want))
