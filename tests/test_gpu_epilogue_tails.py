"""The epilogue's backward pass far out in the activations' tails, up to BF16's
largest value and infinity, against the exact slopes and the float64 oracle."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import workloads
from oracle import step_oracle as so
from tests.test_gpu_epilogue import ACTS, check_backward

pytestmark = pytest.mark.gpu
BIG = float(torch.finfo(torch.bfloat16).max)
FAR = [40.0, 120.0, 1e4, 1e12, 2e13, 1e14, 1.8e19, 1e20, 1e30, BIG, float("inf")]


def place(t, offset):
    """t in rows that begin `offset` elements past a 16-byte boundary."""
    buf = torch.zeros(t.numel() + t.shape[0] * 8 + offset, dtype=t.dtype, device="cuda")
    v = buf[offset:offset + t.shape[0] * (t.shape[1] + 8)].view(t.shape[0], t.shape[1] + 8)[:, :t.shape[1]]
    return v.copy_(t)


@pytest.mark.parametrize("offset", [0, 1])      # 16-byte accesses, element accesses
@pytest.mark.parametrize("act", ACTS)
def test_slopes_in_the_tails(act, offset):
    """Slopes there are 1 and 0, so dz is dy or 0 exactly (but for SiLU's -1.7e-16 at
    -40, off by BF16's rounding and the exponential's 2**-16)."""
    z = torch.tensor(FAR + [-v for v in FAR] + [0.0, -0.0], dtype=torch.bfloat16, device="cuda").repeat(5, 1)
    dy = torch.tensor([1.0, -2.0, 3.0, 0.5, 8.0], dtype=torch.bfloat16, device="cuda")[:, None].expand(z.shape).contiguous()
    slope = torch.cat([torch.ones(len(FAR)), torch.full((len(FAR),), 1.0 if act == "none" else 0.0),
                       torch.full((2,), {"none": 1.0, "relu": 0.0}.get(act, 0.5))]).double()
    if act == "silu":
        slope[len(FAR)] = float(so.act_slope(np.array(-40.0), act))
    slope = slope.cuda()
    dz, dbias = mx.epilogue_backward(place(dy, offset), place(z, offset), act=act)
    exact = slope == (slope * 2).round() / 2
    assert int(exact.sum()) == len(slope) - (act == "silu")
    want = dy.double() * slope
    assert torch.equal(dz.double()[:, exact], want[:, exact])
    assert torch.equal(dbias.double()[exact], want.sum(0)[exact])        # small whole and half numbers: exact sums
    assert ((dz - want).abs() <= (2.0 ** -8 + 2.0 ** -15) * want.abs()).all()
    assert ((dbias - want.sum(0)).abs() <= 2.0 ** -15 * want.abs().sum(0)).all()


@pytest.mark.parametrize("act", ACTS)
def test_every_magnitude(act):
    """z spread over the logarithm of BF16's whole range, either sign."""
    r = workloads.philox(33)
    z = torch.from_numpy((10.0 ** r.uniform(-38, 38.4, (64, 512)) * r.choice([-1.0, 1.0], (64, 512))).astype(np.float32))
    z = z.clamp(-BIG, BIG).cuda().bfloat16()
    dy = workloads.normal_bf16((64, 512), 34).cuda()
    with np.errstate(over="ignore"):
        check_backward(dy, z, act, *mx.epilogue_backward(dy, z, act=act))


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_a_nan_stays_and_stays_alone(act):
    z = torch.full((9, 16), 1e20, dtype=torch.bfloat16, device="cuda")
    z[4, 3] = float("nan")
    dz, dbias = mx.epilogue_backward(torch.ones_like(z), z, act=act)
    nan = torch.isnan(dz)
    assert nan[4, 3] and int(nan.sum()) == 1 and (dz[~nan] == 1).all()
    assert torch.isnan(dbias).nonzero().flatten().tolist() == [3]


def test_the_oracle_is_finite_there():
    for act in ("gelu", "silu"):
        with np.errstate(over="ignore"):
            s = so.act_slope(np.array([1e20, -1e20, 3e38, -3e38]), act)
        assert s.tolist() == [1, 0, 1, 0]
