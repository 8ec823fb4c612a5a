"""The router with more tokens a sequence than there are tokens: the one sequence's
results, bit for bit."""
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
from tests.test_gpu_router import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seq", [501, 1 << 40, (1 << 63) - 500, (1 << 63) - 1])
def test_one_sequence(seq):
    x = make(500, 64, 21)
    dw = torch.randn(500, 6, device="cuda")
    a, b = (mx.router_forward(x, 6, tokens_per_seq=s) for s in (500, seq))
    for f in ("indices", "weights", "counts", "group_offsets", "load", "loss"):
        assert torch.equal(getattr(a, f), getattr(b, f)), f
    assert torch.equal(*(mx.router_backward(x, a.indices, a.load, dw, a.loss, tokens_per_seq=s) for s in (500, seq)))
