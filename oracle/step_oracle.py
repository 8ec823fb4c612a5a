"""CPU oracle of the operators around the products of a training step: AdamW,
layer norm, the epilogue of a product, the router.

Test infrastructure only, plain float64 numpy written from the definitions in
include/mxfp8.h; it shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

STATE_BLOCK = 256


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

def adamw(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step, grad_scale=1.0):
    """One step in float64: (p, m, v, update), update = what the moments took off p."""
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    with np.errstate(invalid="ignore", divide="ignore"):
        update = lr * (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p - lr * weight_decay * p - update, m, v, update


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 E4M3 codes."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7.0))
    mag = np.where((c & 0x7F) == 0x7F, np.nan, mag)
    return np.where(c & 0x80, -mag, mag)


def second_moment_values() -> np.ndarray:
    """The value of each of the 256 codes of the second moment, in units of the
    block's scale: 0, then eighths of binades up to code 255 = 1."""
    out = np.zeros(256)
    for c in range(1, 256):
        out[c] = 2.0 ** ((c + 1) // 8 - 32) * (1 + ((c + 1) % 8) / 8)
    return out


def block_scale(scale, n) -> np.ndarray:
    """One scale for each of n elements."""
    return np.repeat(np.asarray(scale, dtype=np.float64), STATE_BLOCK)[:n]


def block_amax(x) -> np.ndarray:
    x = np.abs(np.asarray(x, dtype=np.float64))
    return np.array([x[i:i + STATE_BLOCK].max() for i in range(0, len(x), STATE_BLOCK)])


# ---------------------------------------------------------------------------
# Layer norm and root-mean-square norm
# ---------------------------------------------------------------------------

def norm_stats(x, eps, center=True):
    mean = x.mean(1) if center else np.zeros(len(x))
    return mean, 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)


def norm(x, w, b, eps, center=True):
    """(y, mean, rstd)."""
    mean, rstd = norm_stats(x, eps, center)
    return (x - mean[:, None]) * rstd[:, None] * w + b, mean, rstd


def norm_backward(dy, x, w, mean, rstd, center=True):
    """(dx, dw, db) from the row statistics."""
    h = (x - mean[:, None]) * rstd[:, None] if center else x * rstd[:, None]
    g = dy * w
    dx = g - h * (g * h).mean(1, keepdims=True)
    if center:
        dx = dx - g.mean(1, keepdims=True)
    return dx * rstd[:, None], (dy * h).sum(0), dy.sum(0)


# ---------------------------------------------------------------------------
# Epilogue of a product: out = act(z) + residual, z = A . B^T + bias
# ---------------------------------------------------------------------------

def act(z, name):
    with np.errstate(over="ignore"):
        if name == "relu":
            return np.where(z > 0, z, 0.0)
        if name == "gelu":
            return 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
        if name == "silu":
            return z / (1 + np.exp(-z))
    return z


def act_slope(z, name):
    with np.errstate(over="ignore"):
        if name == "relu":
            return (z > 0).astype(np.float64)
        if name == "gelu":
            a = np.sqrt(2 / np.pi)
            t = np.tanh(a * (z + 0.044715 * z ** 3))
            return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
        if name == "silu":
            q = 1 / (1 + np.exp(-z))
            return q + z * q * (1 - q)
    return np.ones_like(z)


def epilogue(z, name, residual):
    return act(z, name) + residual


def epilogue_backward(dy, z, name):
    """(dz, dbias)."""
    dz = dy * act_slope(z, name)
    return dz, dz.sum(0)


# ---------------------------------------------------------------------------
# Router: choice, weights, counts, balance loss
# ---------------------------------------------------------------------------

def router_probs(x, mask=None):
    """(p, valid): softmax of each row; rows left out (masked, or no logit above
    -inf) are zero."""
    valid = ~(x == -np.inf).all(1)
    if mask is not None:
        valid &= mask
    y = np.where(valid[:, None], x, 0.0)
    with np.errstate(invalid="ignore"):
        m = np.fmax.reduce(y, axis=1, keepdims=True)
        e = np.exp(y - m)
        p = e / e.sum(1, keepdims=True)
    return np.where(valid[:, None], p, 0.0), valid


def router(x, top_k, seq, mask=None, normalize=False, coef=1.0):
    """dict of indices, weights, counts, offsets, load, loss (and p, valid)."""
    T, E = x.shape
    p, valid = router_probs(x, mask)
    seqs = -(-T // seq)
    idx = np.full((T, top_k), -1)
    w = np.zeros((T, top_k))
    hits = np.zeros((seqs, E), dtype=np.int64)
    for t in range(T):
        if not valid[t]:
            continue
        order = sorted((e for e in range(E) if x[t, e] > -np.inf), key=lambda e: (-x[t, e], e))[:top_k]
        idx[t, :len(order)] = order
        w[t, :len(order)] = p[t, order]
        if normalize:
            w[t] /= p[t, order].sum()
        for e in order:
            hits[t // seq, e] += 1
    n = np.array([valid[s * seq:(s + 1) * seq].sum() for s in range(seqs)])
    psum = np.array([p[s * seq:(s + 1) * seq].sum(0) for s in range(seqs)]).reshape(seqs, E)
    live = max(1, int((n > 0).sum()))
    load = coef * E / (top_k * live) * hits / np.maximum(n, 1)[:, None] ** 2.0
    counts = hits.sum(0)
    return dict(indices=idx, weights=w, counts=counts, offsets=np.concatenate([[0], np.cumsum(counts)]), load=load,
                loss=(load * psum).sum(), p=p, valid=valid, psum=psum)


def router_backward(x, idx, load, dweights, dloss, seq, mask=None, normalize=False):
    p, valid = router_probs(x, mask)
    T, E = x.shape
    g = dloss * load[np.arange(T) // seq]
    for t in range(T):
        if dweights is None or not valid[t]:
            continue
        sel = idx[t][idx[t] >= 0]
        dw = dweights[t][idx[t] >= 0]
        if normalize:
            z = p[t, sel].sum()
            dw = (dw - (dw * p[t, sel] / z).sum()) / z
        g[t, sel] += dw
    dx = p * (g - (p * g).sum(1, keepdims=True))
    return np.where(valid[:, None], dx, 0.0)


# ---------------------------------------------------------------------------
# Gated feed-forward block: the norm with the residual's addition, the gate
# ---------------------------------------------------------------------------

def add_norm(x, residual, w, eps):
    """(sum, rstd, y)."""
    v = x + residual
    rstd = 1.0 / np.sqrt((v * v).mean(1) + eps)
    return v, rstd, v * rstd[:, None] * w


def add_norm_backward(dy, v, w, rstd, dsum):
    """(dx, dw) from the sum and its statistic."""
    h = v * rstd[:, None]
    g = dy * w
    return dsum + rstd[:, None] * (g - h * (g * h).mean(1, keepdims=True)), (dy * h).sum(0)


def gated(gate, up, name):
    return act(gate, name) * up


def gated_backward(dh, gate, up, name):
    """(dgate, dup)."""
    return dh * up * act_slope(gate, name), dh * act(gate, name)


def segments(x, offsets):
    """Rows of x with each group's padded with zeros to a multiple of 128."""
    parts = [np.pad(x[a:b], ((0, -(b - a) % 128), (0, 0))) for a, b in zip(offsets, offsets[1:])]
    return np.concatenate(parts) if parts else x[:0]


def copy_error(codes, scales, ref, tol):
    """How far an MX copy (codes [R, K], logical scales [R, K/32]) of values within
    tol of ref goes beyond what its rounding allows, at most (<= 0: nowhere).

    A block's exponent has to be the one of an amax within tol of ref's; a value may
    be off by half an E4M3 step (2^-4 of it, or 2^-10 of the scale below the normal
    range) and saturates at 448 times the scale."""
    R, K = ref.shape
    val = e4m3_values()[codes].reshape(R, K // 32, 32)
    r, t = np.abs(ref).reshape(val.shape), np.broadcast_to(tol, ref.shape).reshape(val.shape)
    sign_ref = ref.reshape(val.shape)
    X = scales.astype(np.int64) - 127

    def exponent(a):
        with np.errstate(divide="ignore"):
            return np.where(a > 0, np.clip(np.frexp(a)[1] - 1 - 8, -127, 127), -127)

    low, high = exponent(np.maximum(r - t, 0).max(2)), exponent((r + t).max(2))
    worst = np.where((X < low) | (X > high), np.inf, -np.inf).max(initial=-np.inf)
    s = np.exp2(X.astype(np.float64))[..., None]
    room = t + np.maximum((r + t) * 2.0 ** -4, s * 2.0 ** -10)
    return max(worst, (np.abs(val * s - np.clip(sign_ref, -448 * s, 448 * s)) - room).max(initial=-np.inf))
