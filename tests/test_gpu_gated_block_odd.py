"""The dense block where F is no multiple of 128: gate and up of one [2F, C] weight are then
not whole scale atoms, so their row copies are the two matrices of a stacked quantisation,
and the column copy that dgrad reads is the quantiser's of the whole [2F, C]. Against
automatic differentiation in FP32, tolerances as in tests/test_gpu_gated_block.py."""
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
from tests.test_gpu_gated_block import BF16, F32, Dense, normal, off

pytestmark = pytest.mark.gpu


class Any(Dense):
    def __init__(self, C, F, act):
        self.C, self.F, self.act = C, F, act
        self.w = 1.0 + normal((C,), 1, 0.2, F32)
        self.gate_up, self.down = normal((2 * F, C), 2, C ** -0.5), normal((C, F), 3, F ** -0.5)
        rows, _ = mx.quantize_stacked(self.gate_up.view(2, F, C), mx.MX_ROWWISE)
        self.g, self.u = (mx.MXTensor(rows.data[i], rows.scale[i], F, C, mx.MX_ROWWISE) for i in (0, 1))
        _, self.gu_col = mx.quantize(self.gate_up, mx.MX_COLWISE)
        self.d, self.d_col = mx.quantize(self.down)


@pytest.mark.parametrize("T,C,F,act,dtype", [(256, 128, 352, "silu", BF16), (96, 64, 32, "gelu", F32), (160, 352, 160, "silu", F32),
                                             (1024, 2048, 10944, "silu", BF16), (64, 96, 224, "relu", BF16)])
def test_dense_block(T, C, F, act, dtype):
    assert F % 128
    block = Any(C, F, act)
    x, residual, dout = normal((T, C), 5), normal((T, C), 6, 1.0, dtype), normal((T, C), 7, 0.1, dtype)
    st = mx.new_status()
    s, y, dx, dw, dgu, ddown, *copies = block.step(x, residual, dout, status=st)
    assert mx.read_status(st) == 0
    rs, ry, rdx, rdw, rdgu, rddown = block.reference(x, residual, dout)
    assert off(s, rs) < 2.0 ** -8 and off(y, ry) < 0.16
    offs = {"dw": off(dw, rdw), "dgu": off(dgu, rdgu), "ddown": off(ddown, rddown),
            "dx": float((dx.float() - rdx).norm() / (rdx - dout.float()).norm())}
    assert all(v < 0.22 for v in offs.values()), offs


def test_one_token():
    C, F = 2048, 10944
    block = Any(C, F, "silu")
    x, residual = normal((1, C), 5), normal((1, C), 6)
    n = mx.add_norm_quantize(x, residual, block.w, axis=mx.MX_ROWWISE, stats=False)
    h, _ = mx.gemm_gated(n.row, block.g, block.u)
    y = mx.gemm(mx.MX_FPROP, mx.quantize(h, mx.MX_ROWWISE)[0], block.d)
    _, ry, *_ = block.reference(x, residual, residual)
    assert off(y, ry) < 0.16


def test_the_same_bits_from_pass_to_pass():
    """A step's every output, from passes that nothing waits between, other inputs' steps among them."""
    T, C, F = 4096, 1408, 352
    block = Any(C, F, "silu")
    inputs = [(normal((T, C), 10 * i + 5), normal((T, C), 10 * i + 6), normal((T, C), 10 * i + 7, 0.1)) for i in range(2)]
    want = [[t.clone() for t in block.step(*i)] for i in inputs]
    torch.cuda.synchronize()
    for _ in range(6):
        got = [block.step(*inputs[i]) for i in (0, 1, 1, 0)]
        for g, i in zip(got, (0, 1, 1, 0)):
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
