"""The product with bias, activation and residual, and its backward pass,
against float64.

Tolerances. The product is held to the GEMM's own bound before rounding, 1e-6 of
S = sum |a b|, and the bias's addition to 2u of its terms (u = 2**-24); the
activations' slopes are below 1.13, their fast exponential and quotient off by
less than 2**-16 of the result (|u| 2**-23 in the exponent, |u| < 88), and the
BF16 rounding is 2**-8 of the result. A slope z u' q (1 - q) + q is off by 2**-16
of its parts and by the rounding of 1 - q; sums over rows are at most 200
additions in a chain.
"""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import workloads
from oracle import step_oracle as so
from tests.gpu_util import logical_scales

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ACTS = ["none", "relu", "gelu", "silu"]


def f64(t):
    return t.detach().double().cpu().numpy()


def values(t):
    """The exact values of a quantised copy, float64 on the GPU."""
    v = torch.from_numpy(so.e4m3_values()).cuda()[t.data.long()]
    s = torch.from_numpy(np.exp2(logical_scales(t).astype(np.float64) - 127)).cuda()
    return v * s.repeat_interleave(32, 1)[:, :t.k]


def operands(M, N, K, seed, mode=mx.MX_FPROP):
    if mode == mx.MX_WGRAD:
        a = mx.quantize(workloads.normal_bf16((K, M), seed).cuda(), mx.MX_COLWISE)[1]
        b = mx.quantize(workloads.normal_bf16((K, N), seed + 1, K ** -0.5).cuda(), mx.MX_COLWISE)[1]
    elif mode == mx.MX_DGRAD:
        a = mx.quantize(workloads.normal_bf16((M, K), seed).cuda(), mx.MX_ROWWISE)[0]
        b = mx.quantize(workloads.normal_bf16((K, N), seed + 1, K ** -0.5).cuda(), mx.MX_COLWISE)[1]
    else:
        a = mx.quantize(workloads.normal_bf16((M, K), seed).cuda(), mx.MX_ROWWISE)[0]
        b = mx.quantize(workloads.normal_bf16((N, K), seed + 1, K ** -0.5).cuda(), mx.MX_ROWWISE)[0]
    return a, b


def bf16(M, N, seed, pad=0, offset=0):
    buf = torch.full((M * (N + pad) + offset,), float("nan"), dtype=torch.bfloat16, device="cuda")
    t = buf[offset:].view(M, N + pad)[:, :N]
    t.copy_(workloads.normal_bf16((M, N), seed))
    return t


def tact(z, act):
    return torch.from_numpy(so.act(z.cpu().numpy(), act)).cuda()


def check(a, b, out, z, bias, act, residual):
    A, B = values(a), values(b)
    S = A.abs() @ B.abs().T
    ref = A @ B.T
    err = 1e-6 * S
    if bias is not None:
        ref = ref + bias.double()
        err = err + 2 * U * (ref.abs() + bias.double().abs())
    if z is not None:
        bad = (z.double() - ref).abs() > err + 2.0 ** -8 * (ref.abs() + err)
        assert not bad.any(), ("preact", int(bad.sum()))
    y = tact(ref, act)
    err = 1.13 * err + 2.0 ** -16 * y.abs()
    if residual is not None:
        err = err + 2 * U * (y.abs() + residual.double().abs())
        y = y + residual.double()
    bad = ~((out.double() - y).abs() <= err + 2.0 ** -8 * (y.abs() + err))
    assert not bad.any(), ("out", int(bad.sum()), (out.double() - y).abs().max().item())


SHAPES = [(1, 8, 32), (2, 9, 64), (64, 96, 32), (129, 257, 64), (256, 256, 512), (300, 520, 160), (1000, 136, 224),
          (8, 10944, 128), (1500, 4000, 512), (2049, 2311, 96)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(M, N, K, act):
    a, b = operands(M, N, K, M + N)
    bias = torch.from_numpy(workloads.philox(3).standard_normal(N).astype(np.float32)).cuda()
    res = bf16(M, N, 5)
    st = mx.new_status()
    out, z = mx.gemm_epilogue(mx.MX_FPROP, a, b, bias=bias, act=act, residual=res, keep_preact=True, status=st)
    assert mx.read_status(st) == 0
    check(a, b, out, z, bias, act, res)


@pytest.mark.parametrize("mode", [mx.MX_FPROP, mx.MX_DGRAD, mx.MX_WGRAD])
@pytest.mark.parametrize("parts", ["bias", "residual", "preact", ""])
def test_each_part_alone_and_every_mode(mode, parts):
    for M, N, K in ((288, 320, 160), (2560, 2816, 256)):
        a, b = operands(M, N, K, 40, mode)
        bias = torch.from_numpy(workloads.philox(3).standard_normal(N).astype(np.float32)).cuda().bfloat16() if parts == "bias" else None
        res = bf16(M, N, 5) if parts == "residual" else None
        out, z = mx.gemm_epilogue(mode, a, b, bias=bias, act="none", residual=res, keep_preact=parts == "preact")
        check(a, b, out, z, bias, "none", res)
        if res is None and bias is None:
            plain = mx.gemm(mode, a, b)       # the same accumulators, the same rounding
            assert torch.equal(out.view(torch.int16), plain.view(torch.int16))


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("M,N,K", [(200, 300, 64), (2560, 2816, 96)])
def test_pitches_alignment_and_gaps(M, N, K, pad, offset):
    a, b = operands(M, N, K, 50)
    bias = torch.from_numpy(workloads.philox(3).standard_normal(N + 1).astype(np.float32)).cuda()[1:]
    res, out, z = bf16(M, N, 6, pad, offset), bf16(M, N, 7, pad, offset), bf16(M, N, 8, pad, offset)
    mx.gemm_epilogue(mx.MX_FPROP, a, b, bias=bias, act="gelu", residual=res, out=out, preact=z)
    check(a, b, out, z, bias, "gelu", res)
    for t in (out, z):
        if pad:
            gaps = t.as_strided((M - 1, pad), (N + pad, 1), t.storage_offset() + N)
            assert torch.isnan(gaps).all()


@pytest.mark.parametrize("M,N,K", [(200, 304, 64), (2560, 2816, 96)])
def test_residual_in_place(M, N, K):
    a, b = operands(M, N, K, 60)
    res = bf16(M, N, 6)
    out, _ = mx.gemm_epilogue(mx.MX_FPROP, a, b, act="silu", residual=res)
    mine = res.clone()
    mx.gemm_epilogue(mx.MX_FPROP, a, b, act="silu", residual=mine, out=mine)
    assert torch.equal(out.view(torch.int16), mine.view(torch.int16))


def test_empty_sizes():
    a, b = operands(64, 96, 32, 1)
    e = torch.empty((64, 0), dtype=torch.uint8, device="cuda")
    s = torch.empty(0, dtype=torch.uint8, device="cuda")
    a0, b0 = mx.MXTensor(e, s, 64, 0, mx.MX_ROWWISE), mx.MXTensor(torch.empty((96, 0), dtype=torch.uint8, device="cuda"), s, 96, 0, mx.MX_ROWWISE)
    bias, res = torch.linspace(-2, 2, 96, device="cuda"), bf16(64, 96, 2)
    for act in ACTS:
        out, z = mx.gemm_epilogue(mx.MX_FPROP, a0, b0, bias=bias, act=act, residual=res, keep_preact=True)
        ref = so.epilogue(np.broadcast_to(f64(bias), (64, 96)), act, f64(res))
        assert np.abs(f64(out) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-4
        assert torch.equal(z, bias.bfloat16().expand(64, 96))
    none, _ = mx.gemm_epilogue(mx.MX_FPROP, mx.MXTensor(a.data[:0], a.scale, 0, 32, mx.MX_ROWWISE), b, bias=bias)
    assert none.shape == (0, 96)


def test_large_and_not_finite_values():
    """Bias far out in the tails and not finite: the activations saturate, only
    the entries' own columns are touched."""
    a, b = operands(64, 96, 32, 1)
    bias = torch.zeros(96, device="cuda")
    bias[:6] = torch.tensor([1e30, -1e30, 500.0, -500.0, float("inf"), float("nan")])
    for act in ACTS:
        out = mx.gemm_epilogue(mx.MX_FPROP, a, b, bias=bias, act=act)[0].float()
        clean = mx.gemm_epilogue(mx.MX_FPROP, a, b, bias=torch.zeros(96, device="cuda"), act=act)[0].float()
        assert torch.equal(out[:, 6:], clean[:, 6:])
        assert (out[:, 0] > 9e29).all() and (out[:, 4] == float("inf")).all() and torch.isnan(out[:, 5]).all()
        want = (-1e30, -500.0) if act == "none" else (0.0, 0.0)
        assert torch.allclose(out[:, 1], torch.tensor(want[0], device="cuda"), rtol=1e-2)
        assert (out[:, 3] - want[1]).abs().max() < 30 if act == "none" else (out[:, 3] == 0).all()


def check_backward(dy, z, act, dz, dbias):
    fd, fz = f64(dy), f64(z)
    rz, rb = so.epilogue_backward(fd, fz, act)
    if act == "gelu":
        up = 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * fz * fz)
        q = (so.act(fz, act) / np.where(fz == 0, 1, fz))
        q = np.where(fz == 0, 0.5, q)
    elif act == "silu":
        up, q = np.ones_like(fz), 1 / (1 + np.exp(-fz))
    else:
        up, q = np.zeros_like(fz), np.ones_like(fz)
    rounding = 0.0 if act in ("none", "relu") else 1.0
    tol = np.abs(fd) * rounding * (2.0 ** -16 * (q + np.abs(fz * up) * q * (1 - q)) + 8 * U * (1 + np.abs(fz * up) * q))
    bad = np.abs(f64(dz) - rz) > tol + 2.0 ** -8 * (np.abs(rz) + tol) + 1e-38
    assert not bad.any(), ("dz", int(bad.sum()))
    if dbias is not None:
        bad = np.abs(f64(dbias) - rb) > tol.sum(0) + 200 * U * np.abs(rz).sum(0) + 1e-38
        assert not bad.any(), ("dbias", int(bad.sum()))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", [(1, 1), (1, 8), (7, 9), (8, 256), (9, 257), (300, 520), (1000, 136), (8192, 8), (4100, 3000)])
def test_backward(M, N, act):
    dy = bf16(M, N, 70)
    z = bf16(M, N, 71) * 3
    got = mx.epilogue_backward(dy, z, act=act)
    check_backward(dy, z, act, *got)
    for x, y in zip(got, mx.epilogue_backward(dy, z, act=act)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 1), (5, 3)])
def test_backward_pitches_and_parts(pad, offset):
    M, N = 300, 200
    dy, z, dz = (bf16(M, N, 80 + i, pad, offset) for i in range(3))
    got = mx.epilogue_backward(dy, z, act="silu", dz=dz)
    check_backward(dy, z, "silu", *got)
    if pad:
        assert torch.isnan(dz.as_strided((M - 1, pad), (N + pad, 1), dz.storage_offset() + N)).all()
    alone, none = mx.epilogue_backward(dy, z, act="silu", bias_grad=False)
    assert none is None and torch.equal(alone, got[0])
    only = torch.empty(N, device="cuda")
    ws = torch.empty(mx.mx_epilogue_backward_workspace_bytes(M, N), dtype=torch.uint8, device="cuda")
    mx.mx_epilogue_backward(dy.data_ptr(), dy.stride(0), None, 0, M, N, mx.MX_ACT_NONE, None, 0, only.data_ptr(),
                            ws.data_ptr(), ws.numel(), None, torch.cuda.current_stream().cuda_stream)
    check_backward(dy, z, "none", dy, only)


def test_backward_no_rows_and_extreme_values():
    dz, dbias = mx.epilogue_backward(torch.empty((0, 40), dtype=torch.bfloat16, device="cuda"),
                                     torch.empty((0, 40), dtype=torch.bfloat16, device="cuda"), act="gelu")
    assert dz.shape == (0, 40) and (dbias == 0).all()
    z = torch.tensor([[0.0, -0.0, 1e4, -1e4, 300.0, -300.0, 1e-30, -1e-30]], dtype=torch.bfloat16, device="cuda")
    dy = torch.ones_like(z)
    for act, want in (("relu", [0, 0, 1, 0, 1, 0, 1, 0]), ("gelu", [0.5, 0.5, 1, 0, 1, 0, 0.5, 0.5]),
                      ("silu", [0.5, 0.5, 1, 0, 1, 0, 0.5, 0.5])):
        dz, dbias = mx.epilogue_backward(dy, z, act=act)
        assert torch.equal(dz.float().cpu(), torch.tensor([want], dtype=torch.float32)), (act, dz)
        assert torch.allclose(dbias.cpu(), torch.tensor(want, dtype=torch.float32), atol=1e-6)


def test_gradient_against_differences_of_the_forward_pass():
    """d sum(act(z + t v) dy) / dt at 0 through the FP32 bias, whose outputs are
    BF16: the difference over h = 0.25 is off by the roundings (2**-8 of 256 x 64
    outputs, random signs: below 2**-8 * sqrt(16384) / 0.5 = 1) and by h^2/6 of
    the third derivative (below 1 per output, h^2/6 = 0.01 of the sum's size)."""
    M, N, K = 256, 64, 64
    a, b = operands(M, N, K, 90)
    dy = bf16(M, N, 91)
    v = torch.ones(N, device="cuda")
    h = 0.25
    for act in ("gelu", "silu"):
        def loss(t):
            return float((mx.gemm_epilogue(mx.MX_FPROP, a, b, bias=t * v, act=act)[0].double() * dy.double()).sum())
        _, z = mx.gemm_epilogue(mx.MX_FPROP, a, b, bias=0 * v, act=act, keep_preact=True)
        _, db = mx.epilogue_backward(dy, z, act=act)
        num, ana = (loss(h) - loss(-h)) / (2 * h), float(db.double().sum())
        assert abs(num - ana) <= 5 + 0.01 * float(dy.double().abs().sum()), (num, ana)


def test_another_stream_and_a_captured_graph():
    a, b = operands(512, 768, 128, 95)
    bias, res, dy = torch.randn(768, device="cuda"), bf16(512, 768, 96), bf16(512, 768, 97)
    def both():
        out, z = mx.gemm_epilogue(mx.MX_FPROP, a, b, bias=bias, act="gelu", residual=res, keep_preact=True)
        return (out, z, *mx.epilogue_backward(dy, z, act="gelu"))
    ref = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = both()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, cap))


def test_offsets_past_32_bits():
    """An output of more than 2**32 elements, and its backward pass."""
    M, N, K = 2_100_000, 2056, 32
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-200:] = workloads.normal_bf16((200, K), 1).cuda()
    a = mx.quantize(x, mx.MX_ROWWISE)[0]
    b = mx.quantize(workloads.normal_bf16((N, K), 2).cuda(), mx.MX_ROWWISE)[0]
    last = mx.quantize(x[-256:].contiguous(), mx.MX_ROWWISE)[0]
    res = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    res[-1] = 1.0
    out, z = mx.gemm_epilogue(mx.MX_FPROP, a, b, act="silu", residual=res, keep_preact=True)
    want, wz = mx.gemm_epilogue(mx.MX_FPROP, last, b, act="silu", residual=res[-256:].contiguous(), keep_preact=True)
    assert torch.equal(out[-256:], want) and torch.equal(z[-256:], wz) and (out[:1000] == 0).all()
    dz, dbias = mx.epilogue_backward(out, z, act="silu")
    sz, sb = mx.epilogue_backward(want, wz, act="silu")
    assert torch.equal(dz[-256:], sz) and torch.allclose(dbias, sb, rtol=1e-5, atol=1e-5)
