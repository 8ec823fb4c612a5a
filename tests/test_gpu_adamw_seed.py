"""AdamW's random rounding of the 8-bit second moment without a seed of the caller's:
the step count is the seed."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
from tests.test_gpu_adamw import decode8

pytestmark = pytest.mark.gpu


def start(n):
    """Moments of squares up to 2.25, which the first element of each block holds."""
    g = torch.rand(n, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) + 0.5
    g[::256] = 1.5
    p, s = torch.zeros(n, device="cuda"), mx.adamw_state(g, 8)
    mx.adamw_step([p], [g], [s], lr=0.0, betas=(0.0, 0.0), step=1)
    return p, s


def test_second_moment_decays_where_only_the_step_varies():
    """The blocks' first elements keep their gradient, so the scales stay and the
    others' decay by 0.1% a step is the rounding's alone. 1000 steps leave
    0.999**1000 of their mean; a step's rounding adds at most 0.008 (1/8)**2 v**2
    of variance per element, so the mean over 255000 is within 2%."""
    n = 256 * 1000
    p, s = start(n)
    others = np.arange(n) % 256 != 0
    before = decode8(s, n)[1][others].mean()
    g = torch.zeros_like(p)
    g[::256] = 1.5
    for t in range(2, 1002):
        mx.adamw_step([p], [g], [s], lr=0.0, betas=(0.9, 0.999), step=t)
    v = decode8(s, n)[1]
    assert np.allclose(v[~others], 2.25, rtol=1e-3)
    assert abs(v[others].mean() / before / 0.999 ** 1000 - 1) < 0.02, v[others].mean() / before


def test_the_default_is_the_step_count():
    n = 5000
    g = torch.linspace(0.1, 1.0, n, device="cuda")
    codes = []
    for kw in (dict(step=9), dict(step=9, seed=9), dict(step=9, seed=0), dict(step=10)):
        p, s = start(n)
        mx.adamw_step([p], [g], [s], lr=0.0, betas=(0.9, 0.999), **kw)
        codes.append(s.exp_avg_sq.clone())
    assert torch.equal(codes[0], codes[1])
    assert not torch.equal(codes[0], codes[2]) and not torch.equal(codes[0], codes[3])
