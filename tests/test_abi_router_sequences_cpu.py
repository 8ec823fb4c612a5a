"""The router with more tokens a sequence than there are tokens, up to the type's
largest number: one sequence (no GPU needed: sizes and refusals)."""
import os

import pytest

import mxfp8_block_scaled_gb300 as mx
from tests.test_abi_step_cpu import INVALID, SHAPE, router_backward, router_forward

FAR = [101, 1 << 31, 1 << 62, (1 << 63) - 101, (1 << 63) - 100, (1 << 63) - 99, (1 << 63) - 1]


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(mx.LIB_PATH):
        from mxfp8_block_scaled_gb300 import build
        build.build()
    return mx.lib()


@pytest.mark.parametrize("seq", FAR)
def test_workspace_and_checks(seq):
    need = mx.mx_router_workspace_bytes(100, 100, 64)
    assert need == 5 * 64 * 8 + 16 + 16 and mx.mx_router_workspace_bytes(100, seq, 64) == need
    assert router_forward(tokens_per_seq=seq, workspace_bytes=need - 1) == INVALID
    assert router_forward(tokens_per_seq=seq, n_experts=513, ld=513) == SHAPE
    assert router_backward(tokens_per_seq=seq, tokens=1 << 31) == SHAPE
    assert router_backward(tokens_per_seq=seq, tokens=0) == 0


def test_not_positive_ones_are_still_refused():
    for seq in (0, -1, -(1 << 63)):
        for tokens in (0, 100):
            assert router_forward(tokens_per_seq=seq, tokens=tokens) == INVALID
            assert router_backward(tokens_per_seq=seq, tokens=tokens) == INVALID
        assert mx.mx_router_workspace_bytes(100, seq, 64) == 0
