"""What the gated feed-forward block's wrappers allocate belongs to the stream they
are given (no GPU: stand-ins record what happens under which)."""
import inspect

import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
from tests.test_stream_argument_cpu import Side, copy, record, tensor  # noqa: F401 (a fixture)

BF16 = torch.bfloat16
x, z, stat = tensor(64, 96, dtype=BF16), tensor(64, 192, dtype=BF16), tensor(64)

CALLS = {
    "add_norm_quantize": lambda s: mx.add_norm_quantize(x, x, keep_output=True, stream=s),
    "add_norm_backward": lambda s: mx.add_norm_backward(x, x, None, stat, dsum=x, axis=mx.MX_BOTH, stream=s),
    "gemm_gated": lambda s: mx.gemm_gated(copy(64, 32), copy(96, 32), copy(96, 32), keep_preact=True, stream=s),
    "gated_quantize": lambda s: mx.gated_quantize(z, stream=s),
    "gated_backward_quantize": lambda s: mx.gated_backward_quantize(x, z, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocations_belong_to_the_given_stream(name, record):  # noqa: F811
    CALLS[name](Side())
    assert any(what == "empty" for what, _ in record) and any(what == "mx_" + name for what, _ in record)
    assert all(s == Side.cuda_stream for _, s in record), record


@pytest.mark.parametrize("name", CALLS)
def test_without_one_they_belong_to_the_current_stream(name, record):  # noqa: F811
    CALLS[name](None)
    assert record and all(s is None for _, s in record), record


def test_every_wrapper_is_covered():
    from mxfp8_block_scaled_gb300 import gated_block
    have = {n for n, f in vars(gated_block).items() if inspect.isfunction(f) and not n.startswith("_") and f.__module__ == gated_block.__name__}
    assert have == set(CALLS) and have <= set(dir(mx))
    assert all(inspect.signature(getattr(mx, n)).parameters.get("stream") for n in have)
