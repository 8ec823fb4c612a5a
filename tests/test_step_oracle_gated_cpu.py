"""The oracle of the gated feed-forward block, checked on the CPU: gradients
against central differences, the copies' bound against the quantiser's oracle."""
import numpy as np
import pytest

import oracle
from oracle import step_oracle as so
from tests.test_step_oracle_cpu import differences


def rng(seed):
    return np.random.Generator(np.random.Philox(seed))


@pytest.mark.parametrize("shape", [(3, 7), (1, 2), (5, 1)])
def test_add_norm_gradient_against_differences(shape):
    r = rng(5)
    x, res, dy, ds = (r.standard_normal(shape) for _ in range(4))
    w, eps = r.standard_normal(shape[1]), 0.1

    def loss(x_, r_, w_):
        v, _, y = so.add_norm(x_, r_, w_, eps)
        return float((y * dy).sum() + (v * ds).sum())

    v, rstd, _ = so.add_norm(x, res, w, eps)
    dx, dw = so.add_norm_backward(dy, v, w, rstd, ds)
    assert np.allclose(dx, differences(lambda t: loss(t, res, w), x), atol=1e-7)
    assert np.allclose(dx, differences(lambda t: loss(x, t, w), res), atol=1e-7)
    assert np.allclose(dw, differences(lambda t: loss(x, res, t), w), atol=1e-7)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_gated_gradient_against_differences(act):
    r = rng(6)
    g, u, dh = (r.standard_normal((4, 6)) * 2 for _ in range(3))
    dg, du = so.gated_backward(dh, g, u, act)
    assert np.allclose(dg, differences(lambda t: float((so.gated(t, u, act) * dh).sum()), g), atol=1e-7)
    assert np.allclose(du, differences(lambda t: float((so.gated(g, t, act) * dh).sum()), u), atol=1e-7)


def test_segments():
    x = np.arange(10.0).reshape(5, 2)
    s = so.segments(x, [0, 2, 2, 5])
    assert s.shape == (256, 2) and (s[:2] == x[:2]).all() and (s[128:131] == x[2:]).all()
    assert s[2:128].sum() == 0 and s[131:].sum() == 0


def test_copy_error_takes_the_quantiser_and_nothing_else():
    x = rng(7).standard_normal((40, 96)) * np.exp2(rng(8).integers(-20, 20, (40, 3)).repeat(32, 1))
    x[3, :32] = 0
    x[4, 0] = 500 * np.abs(x[4, 1:32]).max()      # saturates
    codes, scales = oracle.mx_quantize_blocks(x.reshape(40, 3, 32))[1].reshape(40, 96), oracle.mx_quantize_rowwise(x)[1]
    assert so.copy_error(codes, scales, x, 0.0) <= 0
    off = scales.copy()
    off[5, 1] += 1
    assert so.copy_error(codes, off, x, 0.0) == np.inf
    wrong = codes.copy()
    wrong[6, 7] ^= 2                              # two steps
    assert so.copy_error(wrong, scales, x, 0.0) > 0
    wrong = codes.copy()
    wrong[6, 7] ^= 0x80
    assert so.copy_error(wrong, scales, x, 0.0) > 0
