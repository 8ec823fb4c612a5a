"""Refusals of the norms' timeout self test (no GPU needed)."""
import os

import pytest

import mxfp8_block_scaled_gb300 as mx
from tests.test_abi_step_cpu import ALIGN, INVALID, status_of


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(mx.LIB_PATH):
        from mxfp8_block_scaled_gb300 import build
        build.build()
    return mx.lib()


def call(**kw):
    d = dict(timeout_ns=2_000_000, dy=0x1000, x=0x2000, rows=4, cols=512, out=0x3000, rstd=0x4000, dweight=0x5000, dbias=0x6000,
             workspace=0x7000, workspace_bytes=4 * 2 * 512 * 4, dev_status=None, stream=None)
    d.update(kw)
    return status_of(mx.mx_selftest_norm_timeout, *d.values())


def test_refusals():
    for bad in (dict(timeout_ns=0), dict(timeout_ns=999_999), dict(timeout_ns=10_000_000_001), dict(rows=0), dict(cols=256),
                dict(cols=16385), dict(x=0), dict(out=0), dict(rstd=0), dict(dweight=0), dict(dbias=0), dict(workspace=0),
                dict(workspace_bytes=4 * 2 * 512 * 4 - 1), dict(dy=0, x=0)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dy=0x1001), dict(x=0x2001), dict(out=0x3001), dict(rstd=0x4002), dict(workspace=0x7008)):
        assert call(**bad) == ALIGN, bad
