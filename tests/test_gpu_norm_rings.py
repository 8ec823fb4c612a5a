"""One warp a row through the ring of shared-memory stages, refilled many hundred times:
no row takes elements of the one that follows it into its stage. Against float64 on the
GPU; the bounds are test_gpu_norm's, with the row's largest magnitudes for the sums."""
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def matrix(rows, cols, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn((rows, cols), device="cuda", generator=g).to(dtype)


def rounding(t):
    return U if t.dtype == torch.float32 else 2.0 ** -8


# widths of one warp a row: forward 257 .. 512 columns, backward 129 .. 256
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [257, 264, 500, 512])
def test_forward(cols, dtype):
    x = matrix(400_000, cols, dtype, cols)
    y, _, rstd = mx.layer_norm(x, center=False)
    for i in range(0, len(x), 50_000):
        d = x[i:i + 50_000].double()
        want = d * (d.square().mean(1, keepdim=True) + 1e-5).rsqrt()
        assert ((y[i:i + 50_000].double() - want).abs() <= (rounding(y) + 120 * U) * want.abs()).all(), i


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [130, 136, 255, 256])
def test_backward(cols, dtype):
    x, dy = matrix(400_000, cols, dtype, cols), matrix(400_000, cols, dtype, cols + 1)
    rstd = torch.linspace(0.5, 2.0, len(x), device="cuda")
    dx, dw, db = mx.layer_norm_backward(dy, x, None, None, rstd, center=False)
    sums, sizes = torch.zeros(2, cols, device="cuda", dtype=torch.float64), torch.zeros(2, cols, device="cuda", dtype=torch.float64)
    for i in range(0, len(x), 50_000):
        d, g, r = x[i:i + 50_000].double(), dy[i:i + 50_000].double(), rstd[i:i + 50_000, None].double()
        h = d * r
        want = r * (g - h * (g * h).mean(1, keepdim=True))
        size = r * (g.abs() + h.abs() * (g * h).abs().mean(1, keepdim=True))
        assert ((dx[i:i + 50_000].double() - want).abs() <= rounding(dx) * want.abs() + 130 * U * size).all(), i
        sums += torch.stack([(g * h).sum(0), g.sum(0)])
        sizes += torch.stack([(g * h).abs().sum(0), g.abs().sum(0)])
    for got, want, size in zip((dw, db), sums, sizes):         # chains of at most 1000 additions
        assert ((got.double() - want).abs() <= 1004 * U * size).all()
