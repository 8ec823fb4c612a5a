"""AdamW over many tensors against the float64 oracle.

Tolerances (u = 2**-24, one FP32 rounding). m is two products and a sum of FP32
values with FP32 constants: at most 4 roundings of terms no larger than
|b1 m| + |c1 g|, the gradient's own scaling one more: 6u of that sum. v has one
more product: 8u of v. p takes two roundings of p and of the update (3u of each),
the constant 1 - lr*wd (u), and the update's approximate quotient and square root
(2**-20 of it together), plus what m's error makes of the update.
"""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import workloads
from oracle import step_oracle as so

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HYPER = dict(lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1, step=7)


def f64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def make(n, seed, grad=torch.float32, size=0.1, offset=0):
    """p, g and FP32 moments of n elements; offset: elements past a 16-byte boundary."""
    r = workloads.philox(seed)
    def t(a, dtype=torch.float32):
        buf = torch.empty(n + offset, dtype=dtype, device="cuda")
        buf[offset:] = torch.from_numpy(a.astype(np.float32)).cuda().to(dtype)
        return buf[offset:]
    p = t(r.standard_normal(n))
    g = t(r.standard_normal(n) * size * 10.0 ** r.integers(-4, 2, n), grad)
    m = t(r.standard_normal(n) * size * 0.3)
    v = t((r.standard_normal(n) * size) ** 2)
    return p, g, m, v


def oracle_step(p, g, m, v, scale=1.0, wd=None, **kw):
    h = {**HYPER, **kw}
    return so.adamw(f64(p), f64(g), m, v, h["lr"], *h["betas"], h["eps"], h["weight_decay"] if wd is None else wd,
                    h["step"], scale)


def check_param(p_new, p_old, g, m_old, ref, scale=1.0, lr=None):
    rp, rm, rv, upd = ref
    lr = HYPER["lr"] if lr is None else lr
    b1 = HYPER["betas"][0]
    m_terms = np.abs(b1 * m_old) + np.abs((1 - b1) * f64(g) * scale)
    ratio = np.divide(np.abs(upd), np.abs(rm), out=np.zeros_like(upd), where=rm != 0)
    tol = 4 * U * np.abs(f64(p_old)) + (3 * U + 2.0 ** -20) * np.abs(upd) + 6 * U * m_terms * ratio + 1e-38
    bad = np.abs(f64(p_new) - rp) > tol
    assert not bad.any(), (int(bad.sum()), np.abs(f64(p_new) - rp).max())


SIZES = [1, 2, 31, 255, 256, 257, 2047, 2048, 2049, 10944, 100003]


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1])
def test_32_bit_states(grad, offset):
    data = [make(n, 100 + i, grad, offset=offset) for i, n in enumerate(SIZES)]
    old = [[t.clone() for t in d] for d in data]
    decay = [0.1 if i % 2 else 0.0 for i in range(len(data))]
    gs = torch.tensor([0.5], device="cuda")
    kw = {**HYPER, "weight_decay": decay}
    mx.adamw_step([d[0] for d in data], [d[1] for d in data], [mx.AdamWState(32, d[2], d[3]) for d in data],
                  grad_scale=gs, **kw)
    for (p, g, m, v), (p0, g0, m0, v0), wd in zip(data, old, decay):
        ref = oracle_step(p0, g0, f64(m0), f64(v0), 0.5, wd=wd)
        terms = np.abs(0.9 * f64(m0)) + np.abs(0.1 * f64(g0) * 0.5)
        assert (np.abs(f64(m) - ref[1]) <= 6 * U * terms + 1e-44).all()
        assert (np.abs(f64(v) - ref[2]) <= 8 * U * ref[2] + 1e-44).all()
        check_param(p, p0, g0, f64(m0), ref, 0.5)
        assert torch.equal(g, g0)


def states8(m, v, seed=3, idx=0):
    """8-bit states that stand for values near m and v, made by a step that keeps them."""
    s = mx.adamw_state(m, 8)
    p = torch.zeros_like(m)
    # beta = 0: m and v become the gradient and its square
    mx.adamw_step([p], [m.clone()], [s], lr=0.0, betas=(0.0, 0.0), seed=seed)
    t = mx.adamw_state(m, 8)
    mx.adamw_step([p], [v.sqrt()], [t], lr=0.0, betas=(0.0, 0.0), seed=seed)
    return mx.AdamWState(8, s.exp_avg, t.exp_avg_sq, s.exp_avg_scale, t.exp_avg_sq_scale)


def decode8(s, n):
    m = so.e4m3_values()[s.exp_avg.view(torch.uint8).cpu().numpy()] * so.block_scale(s.exp_avg_scale.cpu().numpy(), n)
    v = so.second_moment_values()[s.exp_avg_sq.cpu().numpy()] * so.block_scale(s.exp_avg_sq_scale.cpu().numpy(), n)
    return m, v


def check_codes(s, n, rm, rv, m_err, v_err):
    """Stored codes against the exact new moments: m within half a code's step,
    v one of its two neighbours; scales the blocks' largest values. m_err, v_err:
    the FP32 arithmetic's own bound."""
    ms, vs = s.exp_avg_scale.cpu().numpy().astype(np.float64), s.exp_avg_sq_scale.cpu().numpy().astype(np.float64)
    assert (np.abs(ms * 448 - so.block_amax(rm)) <= 4 * U * so.block_amax(rm) + so.block_amax(m_err)).all()
    assert (np.abs(vs - so.block_amax(rv)) <= so.block_amax(v_err)).all()
    m, v = decode8(s, n)
    per = so.block_scale(ms, n)
    with np.errstate(divide="ignore", invalid="ignore"):
        x = np.where(per > 0, np.abs(rm) / per, 0.0)          # in code units
        e = np.maximum(np.floor(np.log2(np.maximum(x, 2.0 ** -20))), -6.0)
    assert (np.abs(m - rm) <= (2.0 ** (e - 4) * (1 + 1e-6) + x * 6 * U) * per + m_err).all()
    per = so.block_scale(vs, n)
    values = so.second_moment_values()
    with np.errstate(divide="ignore", invalid="ignore"):
        f = np.where(per > 0, rv / per, 0.0)
    c = s.exp_avg_sq.cpu().numpy().astype(int)
    assert ((c == 0) == (rv == 0)).all()
    lo, hi = values[np.maximum(c - 1, 0)], values[np.minimum(c + 1, 255)]
    slack = np.divide(v_err, per, out=np.zeros(n), where=per > 0) + 4 * U * f
    ok = (f <= hi + slack) & ((f >= lo - slack) | (c == 1)) | ((c == 255) & (f <= 1 + slack))
    assert ok.all(), np.flatnonzero(~ok)[:5]


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1])
def test_8_bit_states(grad, offset):
    data = [make(n, 300 + i, grad, offset=offset) for i, n in enumerate(SIZES)]
    states = [states8(d[2], d[3]) for d in data]
    if offset:
        def shift(t):
            b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            b[1:] = t
            return b[1:]
        states = [mx.AdamWState(8, shift(s.exp_avg), shift(s.exp_avg_sq), shift(s.exp_avg_scale), shift(s.exp_avg_sq_scale))
                  for s in states]
    before = [decode8(s, d[0].numel()) for s, d in zip(states, data)]
    p0 = [d[0].clone() for d in data]
    mx.adamw_step([d[0] for d in data], [d[1] for d in data], states, seed=11, **HYPER)
    for d, s, (m0, v0), p in zip(data, states, before, p0):
        n = p.numel()
        ref = oracle_step(p, d[1], m0, v0)
        terms = np.abs(0.9 * m0) + np.abs(0.1 * f64(d[1]))
        check_codes(s, n, ref[1], ref[2], 8 * U * terms + 1e-44, 10 * U * ref[2] + 1e-44)
        check_param(d[0], p, d[1], m0, ref)


def test_first_step_from_zero_state():
    p, g, _, _ = make(1000, 1, size=1.0)
    for bits in (32, 8):
        q = p.clone()
        s = mx.adamw_state(q, bits)
        mx.adamw_step([q], [g], [s], **{**HYPER, "step": 1})
        ref = oracle_step(p, g, np.zeros(1000), np.zeros(1000), step=1)
        check_param(q, p, g, np.zeros(1000), ref)


def test_aligned_and_unaligned_tensors_give_the_same_bits():
    n = 5000
    p, g, m, v = make(n, 5)
    s = states8(m, v)
    outs = []
    for off in (0, 1, 3):
        def sh(t):
            b = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
            b[off:] = t
            return b[off:]
        q = [sh(t) for t in (p, g, s.exp_avg, s.exp_avg_sq, s.exp_avg_scale, s.exp_avg_sq_scale)]
        mx.adamw_step([q[0]], [q[1]], [mx.AdamWState(8, *q[2:])], seed=5, **HYPER)
        outs.append([t.clone() for t in (q[0], *q[2:])])
    for o in outs[1:]:
        for a, b in zip(outs[0], o):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch_holds(bits):
    n = 1000
    ps = [torch.full((1 + i % 7,), 1.0 + i, device="cuda") for i in range(n)]
    ps[10] = torch.empty(0, device="cuda")
    gs = [torch.full_like(p, 0.5) for p in ps]
    states = [mx.adamw_state(p, bits) for p in ps]
    mx.adamw_step(ps, gs, states, lr=0.25, step=1)
    for i, p in enumerate(ps):  # the first step moves by lr whatever the gradient's size
        assert torch.allclose(p, torch.full_like(p, 1.0 + i - 0.25), rtol=1e-6, atol=1e-6), i


def test_rounding_of_the_second_moment_is_unbiased_and_seeded():
    """f between two codes: the share rounded up is f's place between them
    (binomial, 6 standard deviations); other seeds give other roundings."""
    n = 256 * 4000
    g = torch.full((n,), 0.7, device="cuda")
    g[::256] = 1.0   # the block's largest: v = 1
    got = []
    for seed in (1, 2):
        p, s = torch.zeros(n, device="cuda"), mx.adamw_state(g, 8)
        mx.adamw_step([p], [g], [s], lr=0.0, betas=(0.0, 0.0), seed=seed)
        got.append(s.exp_avg_sq.clone())
        v = so.second_moment_values()[s.exp_avg_sq.cpu().numpy()]
        v = v[np.arange(n) % 256 != 0]
        x = float(np.float32(0.7)) ** 2     # 0.49: between 0.46875 and 0.5
        assert set(np.unique(v)) == {0.46875, 0.5}
        q = (x - 0.46875) / 0.03125
        assert abs((v == 0.5).mean() - q) <= 6 * np.sqrt(q * (1 - q) / len(v))
    assert not torch.equal(got[0], got[1])


def test_second_moment_decays_in_8_bits():
    """With no gradient v falls by 0.1% a step, less than a code's step: after
    1000 steps its mean is 0.999**1000 of the start's. Each step's rounding adds
    variance below (1/8)**2/4 * v**2 per changed element; over 256000 elements
    the mean is within 2%."""
    n = 256 * 1000
    g = (torch.rand(n, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) + 0.5)
    p, s = torch.zeros(n, device="cuda"), mx.adamw_state(g, 8)
    mx.adamw_step([p], [g], [s], lr=0.0, betas=(0.0, 0.0), seed=1)
    start = decode8(s, n)[1].mean()
    z = torch.zeros_like(g)
    for t in range(1000):
        mx.adamw_step([p], [z], [s], lr=0.0, betas=(0.9, 0.999), seed=100 + t)
    assert abs(decode8(s, n)[1].mean() / start / 0.999 ** 1000 - 1) < 0.02


def test_tiny_and_zero_blocks():
    g = torch.zeros(1024, device="cuda")
    g[256:512] = 1e-35          # m block below 2**-100: zeros; v underflows to 0
    g[512:768] = 1e-18          # v = 1e-36 * c2: kept
    g[768] = -1.0               # the others of the block: m zero, v zero
    p, s = torch.zeros(1024, device="cuda"), mx.adamw_state(g, 8)
    mx.adamw_step([p], [g], [s], lr=1e-3, step=1)
    m, v = decode8(s, 1024)
    assert torch.isfinite(p).all() and np.isfinite(m).all() and np.isfinite(v).all()
    assert (m[:512] == 0).all() and (v[:512] == 0).all()
    assert (v[512:768] > 0).all() and (m[512:768] > 0).all() and m[768] < 0 < v[768]
    assert (m[769:] == 0).all() and (v[769:] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_gradient_stays_in_its_block(bad):
    n = 256 * 4
    p, g, m, v = make(n, 8)
    s = states8(m, v)
    g[300] = bad
    q = p.clone()
    mx.adamw_step([q], [g], [s], seed=1, **HYPER)
    ms, vs = s.exp_avg_scale.cpu().numpy(), s.exp_avg_sq_scale.cpu().numpy()
    assert np.isfinite(ms[[0, 2, 3]]).all() and np.isfinite(vs[[0, 2, 3]]).all()
    assert not np.isfinite(ms[1]) and not np.isfinite(vs[1])
    keep = np.arange(n) != 300
    assert np.isfinite(f64(q)[keep]).all() and np.isnan(f64(q)[300])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_grad_scale_skips_the_step(bits, bad):
    p, g, m, v = make(3000, 9)
    s = mx.AdamWState(32, m, v) if bits == 32 else states8(m, v)
    before = [t.clone() for t in (p, s.exp_avg, s.exp_avg_sq)]
    st = mx.new_status()
    mx.adamw_step([p], [g], [s], grad_scale=torch.tensor([bad], device="cuda"), status=st, **HYPER)
    assert mx.read_status(st) == 5
    for a, b in zip(before, (p, s.exp_avg, s.exp_avg_sq)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
def test_writes_nothing_outside_its_tensors(bits):
    n, pad = 1003, 64
    bufs = [torch.full((n + 2 * pad,), 7.0, device="cuda") for _ in range(2 if bits == 8 else 4)]
    views = [b[pad:pad + n] for b in bufs]
    if bits == 32:
        s = mx.AdamWState(32, views[2].zero_(), views[3].zero_())
        guards = bufs
    else:
        codes = [torch.full((n + 2 * pad,), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.full((4 + 2 * pad,), 7.0, device="cuda") for _ in range(2)]
        s = mx.AdamWState(8, codes[0][pad:pad + n].zero_(), codes[1][pad:pad + n].zero_(), scales[0][pad:pad + 4].zero_(),
                          scales[1][pad:pad + 4].zero_())
        guards = bufs + codes + scales
    views[1].fill_(0.5)
    mx.adamw_step([views[0]], [views[1]], [s], lr=0.1, step=1)
    for b in guards:
        want = 9 if b.dtype == torch.uint8 else 7.0
        assert (b[:pad] == want).all() and (b[-pad:] == want).all()


def test_another_stream_and_a_captured_graph():
    p, g, m, v = make(5000, 12)
    ref = [t.clone() for t in (p, m, v)]
    mx.adamw_step([ref[0]], [g], [mx.AdamWState(32, ref[1], ref[2])], **HYPER)
    mine = [t.clone() for t in (p, m, v)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mx.adamw_step([mine[0]], [g], [mx.AdamWState(32, mine[1], mine[2])], **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, mine))
    cap = [t.clone() for t in (p, m, v)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.adamw_step([cap[0]], [g], [mx.AdamWState(32, cap[1], cap[2])], **HYPER)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, cap))


def test_offsets_past_32_bits():
    """More than 2**32 elements in one tensor: the last ones are updated like a
    short tensor's (the parameter's update does not depend on the rounding)."""
    n = 2 ** 32 + 777
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-777:] = 0.25
    s = mx.adamw_state(p, 8)
    mx.adamw_step([p], [g], [s], lr=0.5, step=1)
    assert (p[-777:] + 0.5).abs().max() < 1e-6 and (p[-2000:-777] == 0).all() and (p[:777] == 0).all()
    assert (s.exp_avg_sq[-777:] > 0).all() and (s.exp_avg_sq[-2000:-777] == 0).all()


def test_minimises_a_quadratic_with_either_states():
    """300 steps on |p - target|^2 / 2: both kinds end within 2% of the start's
    distance, the 8-bit one's path following the 32-bit one's."""
    r = workloads.philox(77)
    target = torch.from_numpy(r.standard_normal(4096).astype(np.float32)).cuda()
    ends = []
    for bits in (32, 8):
        p = torch.zeros(4096, device="cuda")
        s = mx.adamw_state(p, bits)
        for t in range(1, 301):
            mx.adamw_step([p], [p - target], [s], lr=0.05, step=t, seed=t)
        ends.append(float((p - target).norm() / target.norm()))
    assert ends[0] < 0.02 and ends[1] < 0.02, ends


@pytest.mark.parametrize("bits", [32, 8])
def test_no_eps_and_tiny_gradients(bits):
    """eps = 0: the first step moves by lr however small the gradient, down to
    squares below FP32's smallest normal number."""
    g = torch.tensor([1e-3, -1e-10, 1e-17, -3e-19, 1.0], device="cuda")
    p = torch.zeros(5, device="cuda")
    s = mx.adamw_state(p, 32)
    mx.adamw_step([p], [g], [s], lr=0.5, eps=0.0, step=1)
    # v = 0.001 g^2 keeps 23 bits down to 2^-126, then loses them: 1e-17 -> 1e-37, 3e-19 -> 9e-41 (16 bits left)
    assert torch.allclose(p, -0.5 * g.sign(), rtol=1e-4, atol=0), p
    if bits == 8:
        big = torch.full((512,), 1e-2, device="cuda")
        q, t = torch.zeros(512, device="cuda"), mx.adamw_state(big, 8)
        mx.adamw_step([q], [big], [t], lr=0.5, eps=0.0, step=1)
        assert torch.allclose(q, torch.full_like(q, -0.5), rtol=1e-5)
