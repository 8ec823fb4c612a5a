"""The gated feed-forward block put together from its calls, forward and backward, dense
and with routed experts: against automatic differentiation in FP32, and captured,
replayed and given a stream.

Tolerance. An E4M3 operand is off by at most 2**-4 of an element (half a unit in the
last of three fraction bits), 2**-4 / sqrt(3) in the root mean square. A gradient here
depends on at most ten such operands (forward and backward), independent of one
another: sqrt(10) 2**-4 / sqrt(3) = 0.11 of its norm, taken at twice that for the
differences that the norm and the gate form. The block's output depends on five: 0.08,
at twice that 0.16, of the part that the block adds.
"""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import workloads

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def normal(shape, seed, std=1.0, dtype=BF16):
    return torch.from_numpy((workloads.philox(seed).standard_normal(shape) * std).astype(np.float32)).cuda().to(dtype)


class Dense:
    """y = residual stream + down(act(gate(n)) up(n)), n the norm of x + residual."""

    def __init__(self, C, F, act):
        assert F % 128 == 0  # the gate and up rows of one quantised [2F, C] are whole scale atoms
        self.C, self.F, self.act = C, F, act
        self.w = (1.0 + normal((C,), 1, 0.2, F32))
        self.gate_up, self.down = normal((2 * F, C), 2, C ** -0.5), normal((C, F), 3, F ** -0.5)
        self.gu, self.gu_col = mx.quantize(self.gate_up)
        self.d, self.d_col = mx.quantize(self.down)
        half = self.gu.scale.numel() // 2
        self.g, self.u = (mx.MXTensor(self.gu.data[i * F:(i + 1) * F], self.gu.scale[i * half:(i + 1) * half], F, C, mx.MX_ROWWISE)
                          for i in (0, 1))

    def step(self, x, residual, dout, status=None, stream=None):
        """(stream out, gradients) where dout is the gradient of the stream that comes out."""
        kw = dict(status=status, stream=stream)
        n = mx.add_norm_quantize(x, residual, self.w, eps=EPS, **kw)
        _, z = mx.gemm_gated(n.row, self.g, self.u, act=self.act, keep_preact=True, **kw)
        hr, hc = mx.gated_quantize(z, act=self.act, **kw)
        y = mx.gemm(mx.MX_FPROP, hr, self.d, **kw)
        dr, dc = mx.quantize(dout if dout.dtype == BF16 else dout.to(BF16), **kw)
        dh = mx.gemm(mx.MX_DGRAD, dr, self.d_col, **kw)
        ddown = mx.gemm(mx.MX_WGRAD, dc, hc, **kw)
        gr, gc = mx.gated_backward_quantize(dh, z, act=self.act, **kw)
        dn = mx.gemm(mx.MX_DGRAD, gr, self.gu_col, **kw)
        dgu = mx.gemm(mx.MX_WGRAD, gc, n.col, **kw)
        b = mx.add_norm_backward(dn, n.sum, self.w, n.rstd, dsum=dout, axis=mx.MX_BOTH, **kw)
        return [n.sum, y, b.dx, b.dweight, dgu, ddown, b.row.data, b.row.scale, b.col.data, b.col.scale]

    def reference(self, x, residual, dout):
        leaves = [t.detach().float().requires_grad_() for t in (x, residual, self.w, self.gate_up, self.down)]
        fx, fr, w, gu, down = leaves
        s = fx + fr
        n = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * w
        g, u = (n @ gu.T).chunk(2, 1)
        act = {"silu": torch.nn.functional.silu, "gelu": lambda t: torch.nn.functional.gelu(t, approximate="tanh"),
               "relu": torch.relu}[self.act]
        y = (act(g) * u) @ down.T
        (s + y).backward(dout.float())
        return s.detach(), y.detach(), fx.grad, w.grad, gu.grad, down.grad


def off(got, want):
    return float((got.float() - want).norm() / want.norm())


@pytest.mark.parametrize("T,C,F,act,dtype", [(256, 128, 384, "silu", BF16), (96, 64, 128, "gelu", F32), (160, 352, 256, "silu", F32),
                                             (2080, 2048, 1408, "silu", BF16), (32, 32, 128, "relu", BF16)])
def test_dense_block(T, C, F, act, dtype):
    block = Dense(C, F, act)
    x, residual, dout = normal((T, C), 5), normal((T, C), 6, 1.0, dtype), normal((T, C), 7, 0.1, dtype)
    st = mx.new_status()
    s, y, dx, dw, dgu, ddown, *copies = block.step(x, residual, dout, status=st)
    assert mx.read_status(st) == 0
    rs, ry, rdx, rdw, rdgu, rddown = block.reference(x, residual, dout)
    assert off(s, rs) < 2.0 ** -8 and off(y, ry) < 0.16
    offs = {"dw": off(dw, rdw), "dgu": off(dgu, rdgu), "ddown": off(ddown, rddown),
            "dx": float((dx.float() - rdx).norm() / (rdx - dout.float()).norm())}  # of what the block adds to dout
    assert all(v < 0.22 for v in offs.values()), offs


def test_dense_block_of_one_token():
    """What a single token of serving runs: row copies alone, each call's few-row form."""
    C, F = 2048, 1408
    block = Dense(C, F, "silu")
    x, residual = normal((1, C), 5), normal((1, C), 6)
    n = mx.add_norm_quantize(x, residual, block.w, eps=EPS, axis=mx.MX_ROWWISE, stats=False)
    assert n.rstd is None
    h, none = mx.gemm_gated(n.row, block.g, block.u)
    assert none is None
    hr, _ = mx.quantize(h, mx.MX_ROWWISE)
    y = mx.gemm(mx.MX_FPROP, hr, block.d)
    _, ry, *_ = block.reference(x, residual, residual)
    assert off(y, ry) < 0.16


def test_dense_block_captured_and_on_streams():
    """Replays of a captured step on new inputs, and steps given a stream, give an eager step's bits;
    two graphs that replay at the same time do not disturb each other."""
    T, C, F = 320, 256, 384
    block = Dense(C, F, "silu")
    inputs = [(normal((T, C), 10 * i + 5), normal((T, C), 10 * i + 6), normal((T, C), 10 * i + 7, 0.1)) for i in range(4)]
    want = [[t.clone() for t in block.step(*i)] for i in inputs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i, w in zip(inputs, want):
        got = block.step(*i, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w))
    graphs = []
    for _ in range(2):
        held = [t.clone() for t in inputs[0]]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = block.step(*held)
        graphs.append((g, held, out, torch.cuda.Stream()))
    for first, second in ((0, 1), (2, 3), (3, 0)):
        for (g, held, _, s), i in zip(graphs, (first, second)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                for a, b in zip(held, inputs[i]):
                    a.copy_(b)
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for (_, _, out, _), i in zip(graphs, (first, second)):
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


@pytest.mark.parametrize("counts", [[100, 0, 156, 33], [5, 127, 128, 0, 1, 251]])
def test_routed_experts(counts):
    """The same block with an expert for each group of tokens."""
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    E, T, C, F = len(counts), int(offs[-1]), 256, 352
    o, cap = torch.from_numpy(offs).cuda(), mx.mx_grouped_padded_rows(offs)
    w = 1.0 + normal((C,), 1, 0.2, F32)
    gate_up, down = normal((E, 2 * F, C), 2, C ** -0.5, F32), normal((E, C, F), 3, F ** -0.5, F32)
    gu, gu_col = mx.quantize_stacked(gate_up, mx.MX_BOTH)
    d, d_col = mx.quantize_stacked(down, mx.MX_BOTH)
    x, residual, dy = normal((T, C), 5), normal((T, C), 6), normal((T, C), 7, 0.1)
    groups = dict(group_offsets=o, col_capacity=cap)
    st = mx.new_status()
    n = mx.add_norm_quantize(x, residual, w, eps=EPS, axis=mx.MX_ROWWISE, keep_output=True, status=st)
    _, n_col = mx.quantize(n.y, mx.MX_COLWISE, status=st, **groups)
    z = mx.grouped_gemm(mx.MX_FPROP, n.row, gu, o, status=st)
    hr, hc = mx.gated_quantize(z, status=st, **groups)
    y = mx.grouped_gemm(mx.MX_FPROP, hr, d, o, status=st)
    dr, _ = mx.quantize(dy, mx.MX_ROWWISE, status=st)
    _, dc = mx.quantize(dy, mx.MX_COLWISE, status=st, **groups)
    dh = mx.grouped_gemm(mx.MX_DGRAD, dr, d_col, o, status=st)
    ddown = mx.grouped_gemm(mx.MX_WGRAD, dc, hc, o, status=st)
    gr, gc = mx.gated_backward_quantize(dh, z, status=st, **groups)
    dn = mx.grouped_gemm(mx.MX_DGRAD, gr, gu_col, o, status=st)
    dgu = mx.grouped_gemm(mx.MX_WGRAD, gc, n_col, o, status=st)
    b = mx.add_norm_backward(dn, n.sum, w, n.rstd, dsum=dy, status=st)
    assert mx.read_status(st) == 0

    fx, fr, fw, fgu, fd = leaves = [t.detach().float().requires_grad_() for t in (x, residual, w, gate_up, down)]
    s = fx + fr
    fn = s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * fw
    parts = []
    for e in range(E):
        g, u = (fn[offs[e]:offs[e + 1]] @ fgu[e].T).chunk(2, 1)
        parts.append((torch.nn.functional.silu(g) * u) @ fd[e].T)
    fy = torch.cat(parts)
    (s + fy).backward(dy.float())
    assert off(y, fy.detach()) < 0.16
    rdx, _, rdw, rdgu, rddown = (t.grad for t in leaves)
    assert off(b.dweight, rdw) < 0.22
    assert float((b.dx.float() - rdx).norm() / (rdx - dy.float()).norm()) < 0.22
    for e in range(E):
        if counts[e] == 0:
            assert (dgu[e] == 0).all() and (ddown[e] == 0).all()
        else:
            assert off(dgu[e], rdgu[e]) < 0.22 and off(ddown[e], rddown[e]) < 0.22
