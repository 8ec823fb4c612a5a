"""Refusals of the gated block's timeout self test (no GPU needed)."""
import os

import pytest

import mxfp8_block_scaled_gb300 as mx
from tests.test_abi_gated_cpu import INVALID, status_of


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(mx.LIB_PATH):
        from mxfp8_block_scaled_gb300 import build
        build.build()
    return mx.lib()


def test_refusals():
    for what, limit in ((-1, 2_000_000), (3, 2_000_000), (1, 0), (1, 999_999), (2, 10_000_000_001)):
        assert status_of(mx.mx_selftest_block_timeout, what, limit) == INVALID, (what, limit)
    for what, limit in ((1, 1_000_000), (2, 10_000_000_000), (0, 0)):     # the last one takes it back
        assert status_of(mx.mx_selftest_block_timeout, what, limit) == 0
