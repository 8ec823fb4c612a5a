"""The gated feed-forward block: the product with its gate (mx_gemm_gated) and the
gate's quantising calls, against the float64 oracle.

Tolerances (u = 2**-24). Activations: q, the logistic function, is within 2^-16 of
itself, and 1 - q within (1 - q) 2^-16 + 2^-22 (its error vanishes with 1 - q). So
act is off by 2^-15 of itself, and the slope q + z u' q (1 - q) by 2^-15 of (q + |z u'|
q (1 - q)) and 2^-21 |z u'| q. A q below 2^-126 is flushed to zero (2^-125 with its
error): act and slope are then 0, off by all of themselves, |z| q and (1 + |z u'|) q.
Products of BF16 values are exact in FP32, others one rounding each. A product's
accumulators are within 1e-6 of the sum of magnitudes (the GEMM's bound); act moves
by at most 1.13 times what its argument does.
"""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import oracle
import workloads
from oracle import step_oracle as so
from tests.copies import check_copies, check_exact
from tests.gpu_util import f64, u8

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
ACTS = ["none", "relu", "gelu", "silu"]


def normal(rows, cols, seed, std=1.0, pad=0):
    a = workloads.philox(seed).standard_normal((rows, cols)) * std
    buf = torch.full((rows, cols + pad), float("nan"), dtype=BF16, device="cuda")
    t = buf[:, :cols]
    t.copy_(torch.from_numpy(a.astype(np.float32)))
    return t


# --- the product -----------------------------------------------------------

def quantised(rows, k, seed, std):
    t = torch.from_numpy((workloads.philox(seed).standard_normal((rows, k)) * std).astype(np.float32)).to(BF16)
    return mx.quantize(t.cuda(), mx.MX_ROWWISE)[0]


def decoded(t):
    scales = oracle.mx_scale_unswizzle(u8(t.scale), t.rows, t.k // 32)
    return u8(t.data), scales


def check_product(out, pre, a, gate, up, act):
    qa = decoded(a)
    (g, sg), (u, su) = (oracle.mx_gemm_ref(*qa, *decoded(w)) for w in (gate, up))
    ref = so.gated(g, u, act)
    F = gate.rows
    tol = 1.13 * 1e-6 * sg * (np.abs(u) + 1e-6 * su) + np.abs(so.act(g, act)) * 1e-6 * su + 2.0 ** -14 * np.abs(ref)
    got = f64(out)
    bad = ~(np.abs(got - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol))
    assert not bad.any(), ("out", int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:3], ref[bad][:3])
    if pre is not None:
        z = f64(pre)
        for name, got, ref, s in (("gate", z[:, :F], g, sg), ("up", z[:, F:], u, su)):
            bad = ~(np.abs(got - ref) <= 1e-6 * s + 2.0 ** -8 * (np.abs(ref) + 1e-6 * s))
            assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4].tolist())


# tiles: single-CTA and CTA-pair kernels, last columns of 8 to 120, any alignment, one token
@pytest.mark.parametrize("M,F,K,act", [
    (1, 128, 64, "silu"), (1, 1408, 2048, "silu"), (5, 40, 32, "gelu"), (128, 128, 256, "relu"), (130, 136, 96, "none"),
    (333, 1408, 512, "gelu"), (256, 1000, 160, "silu"), (1000, 1376, 2048, "silu"), (2048, 2080, 288, "gelu"), (77, 37, 64, "silu"),
    (300, 1001, 128, "gelu"), (1100, 2499, 64, "relu")])
def test_product(M, F, K, act):
    a, gate, up = quantised(M, K, 1, 1.0), quantised(F, K, 2, 2.0 / K ** 0.5), quantised(F, K, 3, 1.0 / K ** 0.5)
    st = mx.new_status()
    out, pre = mx.gemm_gated(a, gate, up, act=act, keep_preact=True, status=st)
    assert mx.read_status(st) == 0
    check_product(out, pre, a, gate, up, act)
    alone, none = mx.gemm_gated(a, gate, up, act=act)
    assert none is None and torch.equal(alone, out)


# few tokens: every width of the token tile, contractions cut into one to eight, tails of each
@pytest.mark.parametrize("M,F,K,act", [
    (1, 128, 32, "silu"), (16, 1408, 2048, "silu"), (17, 1376, 992, "gelu"), (32, 264, 2048, "relu"), (31, 10944, 128, "silu"),
    (2, 18432, 416, "silu"), (3, 60000, 64, "none"), (9, 333, 7168, "silu"), (33, 520, 2048, "silu"), (64, 1408, 1952, "gelu"),
    (63, 37, 2080, "silu"), (65, 1001, 2048, "silu"), (128, 640, 7168, "relu"), (333, 1408, 2048, "silu"), (385, 130, 4096, "gelu")])
def test_product_of_few_tokens(M, F, K, act):
    test_product(M, F, K, act)


@pytest.mark.parametrize("M", [3, 20, 50, 140])
def test_product_of_few_tokens_pitches(M):
    F, K = 204, 2048
    a, gate, up = quantised(M, K, 7, 1.0), quantised(F, K, 8, 0.1), quantised(F, K, 9, 0.1)
    want, wpre = mx.gemm_gated(a, gate, up, keep_preact=True)
    check_product(want, wpre, a, gate, up, "silu")
    for ldc, ldp, shift in ((208, 416, 0), (203 + 4, 411, 0), (208, 412, 1), (208, 412, 2)):
        c = torch.full((M * ldc + 64,), 7.0, dtype=BF16, device="cuda")
        z = torch.full((M * ldp + 64,), 7.0, dtype=BF16, device="cuda")
        mx.mx_gemm_gated(a.c_operand(), gate.c_operand(), up.c_operand(), mx.MX_ACT_SILU, c.data_ptr() + 2 * shift, ldc,
                         z.data_ptr() + 2 * shift, ldp, None, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        for t, ld, n, ref in ((c, ldc, F, want), (z, ldp, 2 * F, wpre)):
            m = t[shift:shift + M * ld].view(M, ld)
            assert torch.equal(m[:, :n], ref)
            assert (m[:, n:] == 7).all() and (t[:shift] == 7).all() and (t[shift + M * ld:] == 7).all()


def test_product_of_few_tokens_repeats_and_replays():
    """The same bits from every call and from a graph's replays, two of them on two streams at once."""
    F, K = 1408, 2048
    gate, up = quantised(F, K, 8, 0.1), quantised(F, K, 9, 0.1)
    graphs, outs, wants = [], [], []
    tokens = [quantised(M, K, M, 1.0) for M in (1, 48)]  # kept for the graphs' replays
    st = mx.new_status()
    for a in tokens:
        wants.append(mx.gemm_gated(a, gate, up)[0])
        assert torch.equal(mx.gemm_gated(a, gate, up)[0], wants[-1])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                out, _ = mx.gemm_gated(a, gate, up, status=st)
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert mx.read_status(st) == 0
    for got, want in zip(outs, wants):
        assert torch.equal(got, want)


def test_product_of_stacked_weights():
    """The two matrices of one batched quantisation of a weight kept as [2F, K]; F = 1376 is no whole atom."""
    F, K, M = 1376, 320, 512
    w = torch.from_numpy(workloads.philox(5).standard_normal((2, F, K)).astype(np.float32) * 0.06).cuda()
    rows, _ = mx.quantize_stacked(w, mx.MX_ROWWISE)
    gate, up = (mx.MXTensor(rows.data[i], rows.scale[i], F, K, mx.MX_ROWWISE) for i in (0, 1))
    a = quantised(M, K, 6, 1.0)
    out, pre = mx.gemm_gated(a, gate, up, keep_preact=True)
    check_product(out, pre, a, gate, up, "silu")


def test_product_pitches_and_guards():
    M, F, K = 300, 200, 128
    a, gate, up = quantised(M, K, 7, 1.0), quantised(F, K, 8, 0.1), quantised(F, K, 9, 0.1)
    want, wpre = mx.gemm_gated(a, gate, up, keep_preact=True)
    for ldc, ldp, shift in ((208, 416, 0), (203, 405, 0), (208, 408, 1)):
        c = torch.full((M * ldc + 64,), 7.0, dtype=BF16, device="cuda")
        z = torch.full((M * ldp + 64,), 7.0, dtype=BF16, device="cuda")
        mx.mx_gemm_gated(a.c_operand(), gate.c_operand(), up.c_operand(), mx.MX_ACT_SILU, c.data_ptr() + 2 * shift, ldc,
                         z.data_ptr() + 2 * shift, ldp, None, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        for t, ld, n, ref in ((c, ldc, F, want), (z, ldp, 2 * F, wpre)):
            m = t[shift:shift + M * ld].view(M, ld)
            assert torch.equal(m[:, :n], ref)
            assert (m[:, n:] == 7).all() and (t[:shift] == 7).all() and (t[shift + M * ld:] == 7).all()


def test_product_empty_contraction_and_sizes():
    out = torch.full((40, 64), 3.0, dtype=BF16, device="cuda")
    op = lambda rows: mx.MXOperandC(None, None, rows, 0, 0, mx.MX_ROWWISE, 0)  # noqa: E731
    mx.mx_gemm_gated(op(40), op(64), op(64), mx.MX_ACT_SILU, out.data_ptr(), 64, None, 0, None,
                     torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert (out == 0).all()
    gate = quantised(64, 64, 11, 1.0)
    e = torch.empty(0, dtype=torch.uint8, device="cuda")
    none = mx.MXTensor(torch.empty((0, 64), dtype=torch.uint8, device="cuda"), e, 0, 64, mx.MX_ROWWISE)
    out, pre = mx.gemm_gated(none, gate, gate, keep_preact=True)
    assert out.shape == (0, 64) and pre.shape == (0, 128)


# --- the gate's quantising calls --------------------------------------------

def gate_tolerances(dh, g, u, act):
    """(of h, of dgate, of dup)."""
    exact = act in ("none", "relu")
    with np.errstate(over="ignore"):
        if exact:
            s, flushed = np.zeros_like(g), np.zeros(g.shape, dtype=bool)
        else:
            a = 2 * np.sqrt(2 / np.pi)
            v, zu = (g, np.abs(g)) if act == "silu" else (a * (g + 0.044715 * g ** 3), np.abs(a * g * (1 + 3 * 0.044715 * g * g)))
            q = 1 / (1 + np.exp(-v))
            flushed = q < 2.0 ** -125
            s = 2.0 ** -15 * (q + zu * q * (1 - q)) + 2.0 ** -21 * zu * q + np.where(flushed, (1 + zu) * q, 0.0)
    value = np.abs(so.act(g, act)) * (0.0 if exact else np.where(flushed, 1.0, 2.0 ** -15))
    return value * np.abs(u) + 2.0 ** -23 * np.abs(so.gated(g, u, act)), np.abs(dh * u) * (s + 2.0 ** -22), value * np.abs(dh) + \
        2.0 ** -23 * np.abs(so.gated(g, dh, act))


def check_gate(gate_up, dh, act, row, col, brow, bcol, offsets=None):
    F = gate_up.shape[1] // 2
    z, d = f64(gate_up), f64(dh)
    g, u = z[:, :F], z[:, F:]
    th, tg, tu = gate_tolerances(d, g, u, act)
    check_copies(row, col, so.gated(g, u, act), th, "h", offsets)
    check_copies(brow, bcol, np.concatenate(so.gated_backward(d, g, u, act), 1), np.concatenate([tg, tu], 1), "dgate dup", offsets)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,F", [(32, 32), (64, 96), (128, 128), (160, 352), (512, 1408), (96, 10944)])
def test_gate_dense(rows, F, act):
    z, dh = normal(rows, 2 * F, 21, 2.0), normal(rows, F, 22, 0.1)
    st = mx.new_status()
    h = mx.gated_quantize(z, act=act, status=st)
    b = mx.gated_backward_quantize(dh, z, act=act, status=st)
    assert mx.read_status(st) == 0
    check_gate(z, dh, act, *h, *b)


@pytest.mark.parametrize("rows", [1, 3, 31, 33, 127, 130, 1000])
@pytest.mark.parametrize("F,pad", [(32, 0), (224, 8), (1408, 24)])
def test_gate_any_rows_with_pitch(rows, F, pad):
    z, dh = normal(rows, 2 * F, 23, 2.0, pad), normal(rows, F, 24, 0.1, pad)
    h = mx.gated_quantize(z, axis=mx.MX_ROWWISE)
    b = mx.gated_backward_quantize(dh, z, axis=mx.MX_ROWWISE)
    assert h[1] is None and b[1] is None
    check_gate(z, dh, "silu", *h, *b)


@pytest.mark.parametrize("axis", [mx.MX_COLWISE, mx.MX_BOTH])
@pytest.mark.parametrize("counts,F", [([100, 0, 156], 96), ([37, 0, 300, 1, 128], 352), ([0, 0, 129], 64), ([256], 1408), ([0, 5, 0], 32),
                                      ([5, 127, 128, 0, 0, 1000, 33, 2], 224)])
def test_gate_groups(counts, F, axis):
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    M = int(offs[-1])
    z, dh = normal(M, 2 * F, 25, 2.0), normal(M, F, 26, 0.1)
    o = torch.from_numpy(offs).cuda()
    cap = mx.mx_grouped_padded_rows(offs)
    st = mx.new_status()
    h = mx.gated_quantize(z, axis=axis, group_offsets=o, col_capacity=cap, status=st)
    b = mx.gated_backward_quantize(dh, z, axis=axis, group_offsets=o, col_capacity=cap, status=st)
    assert mx.read_status(st) == 0
    check_gate(z, dh, "silu", *h, *b, offsets=offs)
    if axis == mx.MX_BOTH:      # a larger capacity: the same segments, nothing behind them
        big = cap + 256
        col = mx.MXTensor(torch.full((F, big), 0x5A, dtype=torch.uint8, device="cuda"),
                          torch.full((mx.mx_scale_bytes(F, big),), 0x5A, dtype=torch.uint8, device="cuda"), F, big, mx.MX_COLWISE)
        mx.mx_gated_quantize(z.data_ptr(), z.stride(0), M, F, mx.MX_ACT_SILU, mx.MX_COLWISE, None, None, col.data.data_ptr(),
                             col.scale.data_ptr(), o.data_ptr(), len(counts), big, None, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(col.data[:, :cap], h[1].data) and (col.data[:, cap:] == 0x5A).all()
        a = u8(col.scale).reshape(-1, big // 128, 512)
        assert np.array_equal(a[:, :cap // 128], u8(h[1].scale).reshape(-1, cap // 128, 512)) and (a[:, cap // 128:] == 0x5A).all()


@pytest.mark.parametrize("bad", ["order", "end", "start", "capacity"])
def test_gate_bad_offsets_are_reported(bad):
    offs = {"order": [0, 80, 40, 128], "end": [0, 40, 80, 100], "start": [1, 40, 80, 128], "capacity": [0, 40, 80, 128]}[bad]
    z, dh = normal(128, 128, 27), normal(128, 64, 28)
    o = torch.tensor(offs, dtype=torch.int64, device="cuda")
    for back in (False, True):
        width, st = (128 if back else 64), mx.new_status()
        cap = 256 if bad == "capacity" else 384
        col = torch.full((width, cap), 0x5A, dtype=torch.uint8, device="cuda")
        sc = torch.full((mx.mx_scale_bytes(width, cap),), 0x5A, dtype=torch.uint8, device="cuda")
        tail = (None, None, col.data_ptr(), sc.data_ptr(), o.data_ptr(), 3, cap, st.data_ptr(), torch.cuda.current_stream().cuda_stream)
        if back:
            mx.mx_gated_backward_quantize(dh.data_ptr(), 64, z.data_ptr(), 128, 128, 64, mx.MX_ACT_SILU, mx.MX_COLWISE, *tail)
        else:
            mx.mx_gated_quantize(z.data_ptr(), 128, 128, 64, mx.MX_ACT_SILU, mx.MX_COLWISE, *tail)
        assert mx.read_status(st) == 5
        assert (col == 0x5A).all() and (sc == 0x5A).all()


def special_blocks(rows, cols, seed):
    """BF16 values of many magnitudes with zero blocks, negative zeros, subnormals, ties and the largest values."""
    r = workloads.philox(seed)
    a = r.standard_normal((rows, cols)) * np.exp2(r.integers(-40, 40, (rows, cols // 32)).repeat(32, 1).astype(np.float64))
    a[:32, :32] = 0.0
    a[32:64, 5] = -0.0
    a[7, 32:64] = 2.0 ** -130
    a[9, 40] = 3.0e38
    a[:, 33] = np.where(r.random(rows) < 0.5, 1.0625, -1.0625)
    return torch.from_numpy(a.astype(np.float32)).cuda().to(BF16)


@pytest.mark.parametrize("groups", [False, True])
def test_gate_bit_for_bit(groups):
    """With no activation h, dgate and dup are products of two BF16 values, exact in FP32
    (where they neither over- nor underflow): the copies are the quantiser's, byte for byte."""
    rows, F = 224, 160
    g = special_blocks(rows, F, 31)
    r = workloads.philox(32)
    pow2 = np.exp2(r.integers(-4, 4, (rows, F)).astype(np.float64)) * np.where(r.random((rows, F)) < 0.5, -1, 1)
    u = torch.from_numpy((pow2 * (1 + r.integers(0, 128, (rows, F)) / 128)).astype(np.float32)).cuda().to(BF16)
    u[9] = 1.0                                    # 3.0e38 stays finite
    dh = torch.from_numpy(pow2.astype(np.float32)).cuda().to(BF16)
    dh[9] = 1.0
    z = torch.cat([g, u], 1)
    offs = np.array([0, 40, 40, 170, 224]) if groups else None
    kw = dict(group_offsets=torch.from_numpy(offs).cuda(), col_capacity=mx.mx_grouped_padded_rows(offs)) if groups else {}
    fg, fu, fd = f64(g), f64(u), f64(dh)
    check_exact(*mx.gated_quantize(z, act="none", **kw), fg * fu, "h", offs)
    check_exact(*mx.gated_backward_quantize(dh, z, act="none", **kw), np.concatenate([fd * fu, fd * fg], 1), "backward", offs)


def test_gate_not_finite_values():
    """NaN and infinities spoil their own blocks (scale 0xFF, codes 0x7F with each sign) and no other."""
    rows, F = 64, 128
    g, u = special_blocks(rows, F, 33), torch.ones(rows, F, dtype=BF16, device="cuda")
    u[:, ::3] = -1.0
    g[3, 70], g[40, 5], g[41, 100] = float("nan"), float("inf"), float("-inf")
    z = torch.cat([g, u], 1)
    h = f64(g) * f64(u)
    row, col = mx.gated_quantize(z, act="none")
    for copy, v, skip in ((row, h, (3, 70)), (col, h.T, (70, 3))):
        codes, scales = oracle.mx_quantize_rowwise(v)
        got = u8(copy.data).copy()
        # the sign of a NaN product is not defined: that one code's sign bit aside
        assert (got[skip] & 0x7F) == 0x7F
        got[skip] = codes[skip]
        assert np.array_equal(got, codes) and np.array_equal(u8(copy.scale), oracle.mx_scale_swizzle(scales))


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_gate_tails(act):
    """Gates from -1e30 to 1e30: nothing overflows that the function does not."""
    g = torch.tensor([[-1e30, -1e13, -200.0, -90.0, -30.0, -1.0, -0.0, 0.0, 1.0, 30.0, 90.0, 200.0, 1e13, 1e30, 0.5, -0.5] * 2] * 32,
                     dtype=BF16, device="cuda")
    u = torch.full_like(g, 0.5)
    dh = torch.full_like(g, 0.25)
    z = torch.cat([g, u], 1)
    check_gate(z, dh, act, *mx.gated_quantize(z, act=act), *mx.gated_backward_quantize(dh, z, act=act))


def test_gate_full_experts_sampled():
    """The routed experts' size: sampled rows' row copies, and whole segments of some columns."""
    counts = workloads.moe_counts()
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    M, F = int(offs[-1]), 1408
    gen = torch.Generator(device="cuda").manual_seed(5)
    z = torch.randn(M, 2 * F, generator=gen, device="cuda").to(BF16)
    dh = (torch.randn(M, F, generator=gen, device="cuda") * 0.1).to(BF16)
    o, cap = torch.from_numpy(offs).cuda(), mx.mx_grouped_padded_rows(offs)
    row, col = mx.gated_quantize(z, group_offsets=o, col_capacity=cap)
    brow, bcol = mx.gated_backward_quantize(dh, z, group_offsets=o, col_capacity=cap)
    # the dense call on some rows alone gives the same row codes
    pick = torch.tensor(sorted({0, 1, 4097, M // 2, M - 1, *[int(x) for x in offs[:-1] if x < M]}), device="cuda")
    r2, _ = mx.gated_quantize(z[pick].contiguous(), axis=mx.MX_ROWWISE)
    b2, _ = mx.gated_backward_quantize(dh[pick].contiguous(), z[pick].contiguous(), axis=mx.MX_ROWWISE)
    assert torch.equal(row.data[pick], r2.data) and torch.equal(brow.data[pick], b2.data)
    cols = [0, 31, 700, F - 1]
    zg, zu, d = f64(z[:, cols]), f64(z[:, [F + c for c in cols]]), f64(dh[:, cols])
    th, tg, tu = gate_tolerances(d, zg, zu, "silu")
    dg, du = so.gated_backward(d, zg, zu, "silu")
    for copy, at, ref, tol in ((col, cols, so.gated(zg, zu, "silu"), th), (bcol, cols, dg, tg), (bcol, [F + c for c in cols], du, tu)):
        codes = u8(copy.data[at])
        scales = oracle.mx_scale_unswizzle(u8(copy.scale), copy.rows, copy.k // 32)[at]
        assert so.copy_error(codes, scales, so.segments(ref, offs).T, so.segments(tol, offs).T) <= 0


def test_gate_streams_graph_and_bits():
    z, dh = normal(512, 2 * 352, 41), normal(512, 352, 42)

    def step():
        return [t for c in (*mx.gated_quantize(z), *mx.gated_backward_quantize(dh, z)) for t in (c.data, c.scale)]

    want = [t.clone() for t in step()]
    assert all(torch.equal(p, q) for p, q in zip(step(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [t for c in (*mx.gated_quantize(z, stream=side), *mx.gated_backward_quantize(dh, z, stream=side)) for t in (c.data, c.scale)]
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    z2 = normal(512, 2 * 352, 43)
    z.copy_(z2)
    g.replay()
    torch.cuda.synchronize()
    new = [t.clone() for t in held]
    assert all(torch.equal(p, q) for p, q in zip(step(), new))
