"""The epilogue's bias gradient against differences of the forward pass, column by
column, with positive weights dy: nothing cancels, so that the bound is a few
percent of every column's derivative and wrong gradients fall outside it (checked).

Bound of a column's difference [F(h) - F(-h)] / 2h, F(t) = sum over rows of dy
act(z + t): outputs are BF16, each off by 2**-8 of itself at most, hence 2**-8 / h
times sum dy |out|; the third derivative (0.8 at most for both functions) gives h^2/6
of 0.8 sum dy. The kernel's slopes are taken at z rounded to BF16: 2**-8 |z| times
the second derivative (0.8 at most). FP32 sums: 2**-16 of sum dy.
"""
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
from tests.test_gpu_epilogue import bf16, operands

pytestmark = pytest.mark.gpu
M, N, K, H = 1024, 96, 64, 0.125


def column(act):
    """(differences, the kernel's dbias, their bound, sum of dy, the slope's first term alone), each [N]."""
    a, b = operands(M, N, K, 90)
    dy = (bf16(M, N, 91).abs() + 0.5).bfloat16()
    base = torch.linspace(-2.0, 2.0, N, device="cuda")
    w = dy.double()
    out, z = mx.gemm_epilogue(mx.MX_FPROP, a, b, bias=base, act=act, keep_preact=True)
    ends = [mx.gemm_epilogue(mx.MX_FPROP, a, b, bias=base + t, act=act)[0].double() for t in (H, -H)]
    num = (w * (ends[0] - ends[1])).sum(0) / (2 * H)
    _, dbias = mx.epilogue_backward(dy, z, act=act)
    curved = 0.0 if act == "none" else 1.0
    size = (w * torch.maximum(ends[0].abs(), ends[1].abs())).sum(0)
    bound = 2.0 ** -8 / H * size + curved * 0.8 * (H * H / 6 * w.sum(0) + 2.0 ** -8 * (w * z.double().abs()).sum(0)) + 2.0 ** -16 * w.sum(0)
    first = torch.where(z != 0, out.double() / z.double(), 0.5)
    return num, dbias.double(), bound, w.sum(0), (w * first).sum(0)


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_bias_gradient(act):
    num, dbias, bound, _, _ = column(act)
    assert ((num - dbias).abs() <= bound).all(), ((num - dbias).abs() / bound).max()


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_wrong_gradients_fall_outside(act):
    """Most columns refuse no gradient, the opposite one, one a fifth too large, the
    identity's (sum dy) and the slope without its second term."""
    num, dbias, bound, total, first = column(act)
    for wrong in (torch.zeros_like(num), -dbias, 1.2 * dbias, total, first):
        assert ((num - wrong).abs() > bound).double().mean() > 0.5
