"""Layer norm and root-mean-square norm, forward and backward, against the
float64 oracle.

Tolerances (u = 2**-24). A sum over a row's C values is at most 100 additions in
a chain (a thread's own values, then the tree), so it is off by 100u of the sum of
magnitudes; the variance is such a sum of squares of values off by the mean's
error. A sum over rows is at most 200 additions in a chain. A result in BF16 is
rounded once more (8 significant bits: 2**-8 of it).
"""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import workloads
from oracle import step_oracle as so

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ROUND = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
CHAIN, ROWCHAIN = 100, 200


def f64(t):
    return t.detach().double().cpu().numpy()


def matrix(rows, cols, seed, dtype, pad=0, offset=0, mean=0.0, std=1.0):
    a = workloads.philox(seed).standard_normal((rows, cols)) * std + mean
    buf = torch.full((rows * (cols + pad) + offset,), float("nan"), dtype=dtype, device="cuda")
    t = buf[offset:].view(rows, cols + pad)[:, :cols]
    t.copy_(torch.from_numpy(a.astype(np.float32)))
    return t


def vector(cols, seed, dtype, mean=0.0):
    return torch.from_numpy((workloads.philox(seed).standard_normal(cols) * 0.5 + mean).astype(np.float32)).cuda().to(dtype)


def check(got, ref, tol, what):
    got = f64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), np.abs(got - ref)[bad][:3], np.broadcast_to(tol, bad.shape)[bad][:3])


def check_forward(x, w, b, eps, center, y, mean, rstd):
    fx = f64(x)
    fw = f64(w) if w is not None else np.ones(fx.shape[1])
    fb = f64(b) if b is not None else np.zeros(fx.shape[1])
    ry, rm, rr = so.norm(fx, fw, fb, eps, center)
    m_err = CHAIN * U * np.abs(fx).mean(1) if center else np.zeros(len(fx))
    # d = x - mean is off by m_err (the same for a whole row, so the variance by m_err^2) and its own rounding
    d_err = 2 * U * (np.abs(fx).max(1) + np.abs(rm))
    var = 1 / rr ** 2
    v_err = (CHAIN + 4) * U * var + 2 * m_err ** 2 + 2 * d_err * np.sqrt(var) + d_err ** 2
    r_rel = np.minimum(v_err / var, 1.0) + 4 * U
    if center:
        check(mean, rm, m_err + U * np.abs(rm), "mean")
    check(rstd, rr, r_rel * rr, "rstd")
    core = np.abs((fx - rm[:, None]) * rr[:, None] * fw)
    tol = core * (r_rel[:, None] + 6 * U) + np.abs(fw) * ((m_err + d_err) * rr)[:, None] + 2 * U * np.abs(fb)
    check(y, ry, tol + ROUND[y.dtype] * (np.abs(ry) + tol), "y")


# widths around every change of layout: vectors of 8 (BF16) or 4 (FP32), 32 .. 4096 vectors a row, and the looping kernel
WIDTHS = [1, 5, 8, 31, 129, 256, 257, 511, 1009, 1024, 1025, 2048, 2051, 4097, 7168, 8192, 16384, 16392, 33000]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", WIDTHS)
def test_forward_widths(cols, dtype):
    for center, pad in ((True, 0), (False, 8)):
        x = matrix(5, cols, cols, dtype, pad)
        w, b = vector(cols, 1, torch.float32, 1.0), vector(cols, 2, torch.float32)
        y, mean, rstd = mx.layer_norm(x, w, b, eps=1e-5, center=center)
        assert (mean is None) == (not center)
        check_forward(x, w, b, 1e-5, center, y, mean, rstd)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols,rows", [(40, 5000), (2048, 700), (7168, 400)])
def test_forward_many_rows(cols, rows, dtype):
    x = matrix(rows, cols, 7, dtype)
    w, b = vector(cols, 1, torch.bfloat16, 1.0), vector(cols, 2, torch.bfloat16)
    check_forward(x, w, b, 1e-6, True, *mx.layer_norm(x, w, b, eps=1e-6))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 2), (8, 0)])
def test_forward_pitches_and_alignment(pad, offset, dtype):
    x = matrix(9, 1000, 3, dtype, pad, offset)
    y, mean, rstd = mx.layer_norm(x, eps=1e-5)
    check_forward(x, None, None, 1e-5, True, y, mean, rstd)
    out = matrix(9, 1000, 4, dtype, pad, offset)
    mx.layer_norm(x, eps=1e-5, out=out)
    assert torch.equal(out, y)
    whole = out.as_strided((9 * (1000 + pad) - pad,), (1,))
    gaps = torch.ones(whole.numel(), dtype=torch.bool)
    for r in range(9):
        gaps[r * (1000 + pad):r * (1000 + pad) + 1000] = False
    assert torch.isnan(whole[gaps.cuda()]).all()      # the pitch gaps are not written


def test_forward_mean_much_larger_than_spread():
    """x = 1000 + N(0, 1) in FP32: the centred second sweep keeps the variance."""
    x = matrix(64, 4096, 9, torch.float32, mean=1000.0)
    check_forward(x, None, None, 0.0, True, *mx.layer_norm(x, eps=0.0))


def test_constant_zero_and_not_finite_rows():
    x = matrix(6, 300, 11, torch.float32)
    x[1] = 3.0
    x[2] = 0.0
    x[3, 17] = float("nan")
    x[4, 20] = float("inf")
    y, mean, rstd = mx.layer_norm(x, eps=1e-5)
    assert (y[1:3] == 0).all() and torch.allclose(rstd[1:3], torch.full((2,), 1e-5 ** -0.5, device="cuda"))
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    ok = x[[0, 5]].clone()
    assert torch.equal(mx.layer_norm(ok, eps=1e-5)[0], y[[0, 5]])     # the other rows are untouched by them


def test_no_rows_and_no_statistics():
    x = torch.empty((0, 64), device="cuda")
    y, mean, rstd = mx.layer_norm(x)
    assert y.shape == (0, 64)
    dx, dw, db = mx.layer_norm_backward(y, x, None, mean, rstd)
    assert (dw == 0).all() and (db == 0).all() and dw.numel() == 64
    x = matrix(4, 64, 1, torch.float32)
    y, mean, rstd = mx.layer_norm(x, stats=False)
    assert mean is None and rstd is None and torch.equal(y, mx.layer_norm(x)[0])


def check_backward(dy, x, w, mean, rstd, center, dx, dw, db):
    fx, fd, fr = f64(x), f64(dy), f64(rstd)
    fm = f64(mean) if center else np.zeros(len(fx))
    fw = f64(w) if w is not None else np.ones(fx.shape[1])
    rx, rw, rb = so.norm_backward(fd, fx, fw, fm, fr, center)
    h = (fx - fm[:, None]) * fr[:, None]
    h_err = 2 * U * (np.abs(fx) + np.abs(fm)[:, None]) * fr[:, None]
    g = fd * fw
    s1 = np.abs(g).mean(1, keepdims=True)
    s2 = np.abs(g * h).mean(1, keepdims=True) + np.abs(g * h_err).mean(1, keepdims=True)
    e1, e2 = (CHAIN + 4) * U * s1, (CHAIN + 6) * U * s2 + np.abs(g * h_err).mean(1, keepdims=True)
    tol = fr[:, None] * (e1 * center + np.abs(h) * e2 + h_err * s2 + 8 * U * (np.abs(g) + s1 + np.abs(h) * s2))
    check(dx, rx, tol + ROUND[dx.dtype] * (np.abs(rx) + tol), "dx")
    if dw is not None:
        check(dw, rw, ((ROWCHAIN + 4) * U * np.abs(fd * h) + np.abs(fd) * h_err).sum(0) + 1e-38, "dweight")
        check(db, rb, ROWCHAIN * U * np.abs(fd).sum(0), "dbias")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", WIDTHS)
def test_backward_widths(cols, dtype):
    for center, pad, wd in ((True, 0, torch.float32), (False, 8, torch.bfloat16)):
        x, dy = matrix(5, cols, cols, dtype, pad, mean=0.3), matrix(5, cols, cols + 1, dtype, pad)
        w = vector(cols, 1, wd, 1.0)
        _, mean, rstd = mx.layer_norm(x, w, center=center)
        check_backward(dy, x, w, mean, rstd, center, *mx.layer_norm_backward(dy, x, w, mean, rstd, center=center))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols,rows", [(3, 20000), (40, 5000), (256, 3000), (512, 3000), (1024, 2000), (2048, 1500),
                                       (4096, 700), (7168, 400), (16384, 320), (33000, 310)])
def test_backward_many_rows(cols, rows, dtype):
    x, dy = matrix(rows, cols, 7, dtype, mean=0.3), matrix(rows, cols, 8, dtype)
    w = vector(cols, 1, torch.float32, 1.0)
    _, mean, rstd = mx.layer_norm(x, w)
    got = mx.layer_norm_backward(dy, x, w, mean, rstd)
    check_backward(dy, x, w, mean, rstd, True, *got)
    for a, b in zip(got, mx.layer_norm_backward(dy, x, w, mean, rstd)):   # the same bits every time
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 2)])
def test_backward_pitches_and_alignment(pad, offset, dtype):
    x, dy = matrix(700, 1000, 3, dtype, pad, offset), matrix(700, 1000, 4, dtype, pad, offset)
    w = vector(1001, 5, torch.float32, 1.0)[1:]
    _, mean, rstd = mx.layer_norm(x, w.clone())
    check_backward(dy, x, w, mean, rstd, True, *mx.layer_norm_backward(dy, x, w, mean, rstd))
    dx, dw, db = mx.layer_norm_backward(dy, x, None, mean, rstd, param_grads=False)
    assert dw is None and db is None
    check_backward(dy, x, None, mean, rstd, True, dx, None, None)


def test_gradient_against_differences_of_the_forward_pass():
    """Directional derivative of sum(y * dy) along random directions, FP32:
    central differences with step h are off by h^2 (third derivatives of order
    1 here) and by the forward pass's rounding over h: 1e-4 + 1e-6/1e-2."""
    x, dy = matrix(16, 96, 21, torch.float32), matrix(16, 96, 22, torch.float32)
    w, b = vector(96, 23, torch.float32, 1.0), vector(96, 24, torch.float32)
    _, mean, rstd = mx.layer_norm(x, w, b, eps=0.1)
    dx, dw, db = mx.layer_norm_backward(dy, x, w, mean, rstd)
    h = 1e-2
    loss = lambda x_, w_, b_: float((mx.layer_norm(x_, w_, b_, eps=0.1)[0].double() * dy.double()).sum())  # noqa: E731
    for seed in range(3):
        vx, vw, vb = (torch.randn(t.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)) for t in (x, w, b))
        num = (loss(x + h * vx, w + h * vw, b + h * vb) - loss(x - h * vx, w - h * vw, b - h * vb)) / (2 * h)
        ana = float((dx.double() * vx).sum() + (dw.double() * vw).sum() + (db.double() * vb).sum())
        size = float((dx.double() * vx).abs().sum() + (dw.double() * vw).abs().sum() + (db.double() * vb).abs().sum())
        assert abs(num - ana) <= 1e-3 * size, (num, ana)


def test_offsets_past_32_bits():
    """Rows more than 2**32 elements apart."""
    rows, cols = 600_000, 7200
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    last = matrix(2, cols, 31, torch.bfloat16)
    x[-2:] = last
    y, mean, rstd = mx.layer_norm(x)
    assert torch.equal(y[-2:], mx.layer_norm(last)[0]) and (y[-1000:-2] == 0).all()
    dx, dw, db = mx.layer_norm_backward(x, x, None, mean, rstd)
    small = mx.layer_norm_backward(last, last, None, mean[-2:].clone(), rstd[-2:].clone())
    assert torch.equal(dx[-2:], small[0])
    check_backward(last, last, None, mean[-2:], rstd[-2:], True, small[0], dw, db)


def test_another_stream_and_a_captured_graph():
    x, dy = matrix(100, 512, 41, torch.bfloat16), matrix(100, 512, 42, torch.bfloat16)
    w = vector(512, 1, torch.float32, 1.0)
    def both():
        y, mean, rstd = mx.layer_norm(x, w)
        return (y, *mx.layer_norm_backward(dy, x, w, mean, rstd))
    ref = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = both()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, cap))


# Narrow rows: around every number of lanes a row takes, in vectors (of 8 or 4) and in elements.
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [2, 4, 7, 9, 16, 17, 24, 32, 33, 40, 63, 64, 65, 72, 96, 127, 128, 130, 136, 192, 250, 255])
def test_narrow_rows(cols, dtype):
    rows = 777
    for pad, offset, center, pd in ((0, 0, True, torch.float32), (8, 0, False, torch.bfloat16), (1, 3, True, torch.bfloat16)):
        x, dy = matrix(rows, cols, cols, dtype, pad, offset, mean=0.5), matrix(rows, cols, cols + 1, dtype, pad, offset)
        w, b = vector(cols, 1, pd, 1.0), vector(cols, 2, pd)
        out = matrix(rows, cols, 4, dtype, pad, offset)
        y, mean, rstd = mx.layer_norm(x, w, b, center=center, out=out)
        check_forward(x, w, b, 1e-5, center, y, mean, rstd)
        if pad:
            whole = out.as_strided((rows, cols + pad), (cols + pad, 1))[:-1, cols:]
            assert torch.isnan(whole).all()      # the gaps are not written
        got = mx.layer_norm_backward(dy, x, w, mean, rstd, center=center)
        check_backward(dy, x, w, mean, rstd, center, *got)
        for p, q in zip(got, mx.layer_norm_backward(dy, x, w, mean, rstd, center=center)):
            assert torch.equal(p, q)
        dx, dw, db = mx.layer_norm_backward(dy, x, None, mean, rstd, center=center, param_grads=False)
        check_backward(dy, x, None, mean, rstd, center, dx, None, None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols,rows", [(1, 1), (64, 1), (128, 33), (13, 60001), (128, 40000)])
def test_narrow_rows_few_and_many(cols, rows, dtype):
    x, dy = matrix(rows, cols, 3, dtype, mean=-0.2), matrix(rows, cols, 4, dtype)
    w, b = vector(cols, 1, torch.float32, 1.0), vector(cols, 2, torch.float32)
    y, mean, rstd = mx.layer_norm(x, w, b)
    check_forward(x, w, b, 1e-5, True, y, mean, rstd)
    check_backward(dy, x, w, mean, rstd, True, *mx.layer_norm_backward(dy, x, w, mean, rstd))
