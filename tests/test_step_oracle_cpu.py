"""The oracle of the operators around the products, checked against itself on
the CPU: gradients against central differences, codes against their listing."""
import numpy as np
import pytest

from oracle import step_oracle as so


def differences(f, x, h=1e-5):
    """Gradient of the scalar f by central differences (error ~ h^2 and eps/h: 1e-9 here)."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("shape", [(3, 7), (1, 2), (5, 1)])
def test_norm_gradient_against_differences(center, shape):
    r = np.random.Generator(np.random.Philox(5))
    x, dy = r.standard_normal(shape), r.standard_normal(shape)
    w, b = r.standard_normal(shape[1]), r.standard_normal(shape[1])
    eps = 0.1
    mean, rstd = so.norm_stats(x, eps, center)
    dx, dw, db = so.norm_backward(dy, x, w, mean, rstd, center)
    loss = lambda x_, w_, b_: float((so.norm(x_, w_, b_, eps, center)[0] * dy).sum())  # noqa: E731
    assert np.allclose(dx, differences(lambda t: loss(t, w, b), x), atol=1e-7)
    assert np.allclose(dw, differences(lambda t: loss(x, t, b), w), atol=1e-7)
    assert np.allclose(db, differences(lambda t: loss(x, w, t), b), atol=1e-7)


def test_second_moment_codes():
    v = so.second_moment_values()
    assert v[0] == 0 and v[255] == 1 and v[254] == 0.9375 and v[247] == 0.5 and v[1] == 2.0 ** -32 * 1.25
    assert (np.diff(v) > 0).all()
    assert (v[2:] / v[1:-1] <= 1.125).all() and (v[2:] / v[1:-1] >= 16 / 15 - 1e-12).all()


def test_adamw_closed_forms():
    # the first step moves by lr against the gradient's sign; decay is decoupled
    p, m, v, u = so.adamw(np.array([1.0, 1.0]), np.array([3.0, -1e-3]), np.zeros(2), np.zeros(2), 0.1, 0.9, 0.999, 0.0, 0.5, 1)
    assert np.allclose(u, [0.1, -0.1]) and np.allclose(p, 1 - 0.05 - u)
    assert np.allclose(m, [0.3, -1e-4]) and np.allclose(v, [9e-3, 1e-9])


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu"])
def test_epilogue_gradient_against_differences(name):
    r = np.random.Generator(np.random.Philox(6))
    z, dy, b = r.standard_normal((4, 5)) * 2, r.standard_normal((4, 5)), r.standard_normal(5)
    z = z + np.sign(z) * 0.01     # away from relu's corner
    dz, db = so.epilogue_backward(dy, z, name)
    loss = lambda z_, b_: float((so.epilogue(z_ + b_ - b, name, 1.0) * dy).sum())  # noqa: E731
    assert np.allclose(dz, differences(lambda t: loss(t, b), z), atol=1e-7)
    assert np.allclose(db, differences(lambda t: loss(z, t), b), atol=1e-7)


@pytest.mark.parametrize("normalize", [False, True])
def test_router_gradient_against_differences(normalize):
    r = np.random.Generator(np.random.Philox(7))
    x, dw = r.standard_normal((6, 5)) * 2, r.standard_normal((6, 2))
    x[1, 3] = -np.inf
    mask = np.array([1, 1, 0, 1, 1, 1], dtype=bool)
    f = so.router(x, 2, 4, mask, normalize, 0.7)
    dx = so.router_backward(x, f["indices"], f["load"], dw, 1.3, 4, mask, normalize)

    def loss(t):     # the choice and the load are constants
        g = so.router(t, 2, 4, mask, normalize, 0.7)
        assert (g["indices"] == f["indices"]).all()
        return float((g["weights"] * dw).sum() + 1.3 * (f["load"] * g["psum"]).sum())

    num = differences(loss, np.where(np.isinf(x), -50.0, x))
    assert np.allclose(dx, num, atol=1e-7)
    assert (dx[2] == 0).all() and dx[1, 3] == 0


def test_router_balance_closed_forms():
    # every token spread evenly, choices even: loss = coef
    x = np.zeros((4, 4))
    x[np.arange(4), np.arange(4)] = 1e-9
    f = so.router(x, 1, 4, coef=0.3)
    assert np.isclose(f["loss"], 0.3) and (f["counts"] == 1).all() and (f["offsets"] == np.arange(5)).all()
    # all tokens to one expert with certainty: loss = coef * E
    x = np.zeros((4, 4))
    x[:, 2] = 100.0
    assert np.isclose(so.router(x, 1, 2, coef=0.3)["loss"], 1.2)
