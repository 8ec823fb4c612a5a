"""The 8-bit second moment of blocks whose largest value is below FP32's smallest
normal number: the codes keep the elements' ratios."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import workloads
from oracle import step_oracle as so
from tests.test_gpu_adamw import check_codes

pytestmark = pytest.mark.gpu


def moments(g, offset):
    """State after one step that takes g^2 as it is; `offset`: bytes and elements past the aligned places."""
    n = len(g)
    def room(dtype, size=n):
        return torch.zeros(size + offset, dtype=dtype, device="cuda")[offset:]
    p, gt = room(torch.float32), room(torch.float32).copy_(torch.from_numpy(g))
    s = mx.AdamWState(8, room(torch.uint8), room(torch.uint8), *(torch.zeros(-(-n // 256), device="cuda") for _ in range(2)))
    mx.adamw_step([p], [gt], [s], lr=0.0, betas=(0.0, 0.0), step=1)
    return s


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("e", [-62, -63, -64, -65, -70])      # the largest g is 2^e, its square down to 2^-140
def test_powers_of_two_are_exact(e, offset):
    """Squares 1, 1/4, 1/16, 1/64 and 1/256 of the block's largest have codes of their own."""
    k = np.arange(512) % 5
    s = moments((2.0 ** (e - k)).astype(np.float32), offset)
    assert (s.exp_avg_sq_scale.cpu().numpy() == np.float32(2.0 ** (2 * e))).all()
    assert np.array_equal(s.exp_avg_sq.cpu().numpy(), 255 - 16 * k)


@pytest.mark.parametrize("offset", [0, 1])
def test_neighbouring_codes_and_zeros(offset):
    """Any values: each code is one of its value's two neighbours (FP32 keeps g^2 within 2^-150)."""
    r = workloads.philox(5)
    g = (r.standard_normal(2048) * 2.0 ** np.repeat([-60, -63, -64, -65, -66, -68, -70, -72], 256)).astype(np.float32)
    g[::9] = 0.0
    v = g.astype(np.float64) ** 2
    s = moments(g, offset)
    sq = v.astype(np.float32).astype(np.float64)           # what FP32 can hold
    m = np.where(np.repeat(so.block_amax(g), 256) < 2.0 ** -100, 0.0, g.astype(np.float64))
    check_codes(s, len(g), m, sq, np.abs(m) * 2.0 ** -22, sq * 2.0 ** -22 + 2.0 ** -149)
