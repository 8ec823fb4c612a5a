"""Host-side refusals of the gated feed-forward block's calls (no GPU needed)."""
import os

import pytest
import torch

import mxfp8_block_scaled_gb300 as mx

INVALID, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(mx.LIB_PATH):
        from mxfp8_block_scaled_gb300 import build
        build.build()
    return mx.lib()


def status_of(fn, *args):
    try:
        fn(*args)
    except mx.MXError as e:
        return e.status
    return 0


COPIES = dict(row_data=0x10000, row_scale=0x20000, col_data=0x30000, col_scale=0x40000)


def forward(**kw):
    d = dict(x=0x1000, ldx=64, residual=0x2000, ld_residual=64, stream_dtype=mx.MX_BF16, weight=0x3000, param_dtype=mx.MX_F32,
             rows=32, cols=64, eps=1e-5, axis=mx.MX_BOTH, sum=0x4000, ld_sum=64, y=0x5000, ldy=64, rstd=0x6000, **COPIES,
             dev_status=None, stream=None)
    d.update(kw)
    return status_of(mx.mx_add_norm_quantize, *d.values())


def test_add_norm_refusals():
    assert forward(rows=0) == 0
    assert forward(rows=0, axis=0, y=None) == 0
    for bad in (dict(rows=-1), dict(cols=0), dict(stream_dtype=2), dict(param_dtype=-1), dict(axis=-1), dict(axis=4),
                dict(eps=-1.0), dict(eps=float("inf")), dict(x=0), dict(ldx=63), dict(ld_residual=56), dict(ld_sum=56),
                dict(ldy=56), dict(row_data=None), dict(col_scale=None), dict(axis=0, y=None)):
        assert forward(**bad) == INVALID, bad
    for bad in (dict(cols=48), dict(rows=33), dict(cols=16416, ldx=16416), dict(rows=1 << 31)):
        assert forward(**bad) == SHAPE, bad
    for bad in (dict(x=0x1008), dict(ldx=68), dict(residual=0x2002), dict(ld_residual=68), dict(sum=0x4008), dict(y=0x5004),
                dict(weight=0x3002), dict(rstd=0x6002), dict(row_scale=0x20004), dict(col_data=0x30008),
                dict(stream_dtype=mx.MX_F32, ld_residual=66)):
        assert forward(**bad) == ALIGN, bad


def backward(**kw):
    d = dict(dy=0x1000, lddy=64, sum=0x2000, ld_sum=64, dsum=0x3000, ld_dsum=64, stream_dtype=mx.MX_BF16, weight=0x4000,
             param_dtype=mx.MX_F32, rstd=0x5000, rows=32, cols=64, axis=mx.MX_BOTH, dx=0x6000, lddx=64, dweight=0x7000, **COPIES,
             workspace=0x8000, workspace_bytes=1 << 20, dev_status=None, stream=None)
    d.update(kw)
    return status_of(mx.mx_add_norm_backward, *d.values())


def test_add_norm_backward_refusals():
    assert backward(rows=0, dweight=None) == 0
    for bad in (dict(rows=-1), dict(cols=0), dict(stream_dtype=-1), dict(axis=4), dict(dy=0), dict(sum=0), dict(rstd=None),
                dict(lddy=56), dict(ld_sum=56), dict(ld_dsum=56), dict(lddx=56), dict(dx=None, axis=0), dict(row_scale=None),
                dict(col_data=None), dict(workspace=None), dict(workspace_bytes=255)):
        assert backward(**bad) == INVALID, bad
    for bad in (dict(cols=80), dict(rows=40), dict(cols=16416)):
        assert backward(**bad) == SHAPE, bad
    for bad in (dict(dy=0x1002), dict(sum=0x2008), dict(dsum=0x3004), dict(dx=0x6008), dict(dweight=0x7002), dict(rstd=0x5001),
                dict(workspace=0x8008), dict(lddx=68), dict(col_scale=0x40008)):
        assert backward(**bad) == ALIGN, bad
    assert mx.mx_add_norm_backward_workspace_bytes(32, 64) == 64 * 4
    assert mx.mx_add_norm_backward_workspace_bytes(33, 64) == 2 * 64 * 4
    assert mx.mx_add_norm_backward_workspace_bytes(1 << 20, 64) == 608 * 64 * 4
    assert mx.mx_add_norm_backward_workspace_bytes(0, 64) == 0


def operand(data=0x10000, scale=0x20000, rows=128, k=256, ld=0, orient=mx.MX_ROWWISE):
    return mx.MXOperandC(data, scale, rows, k, ld, orient, 0)


def product(a=None, gate=None, up=None, **kw):
    d = dict(act=mx.MX_ACT_SILU, c=0x40000, ldc=128, preact=0x50000, ld_preact=256, dev_status=None, stream=None)
    d.update(kw)
    return status_of(mx.mx_gemm_gated, a or operand(), gate or operand(), up or operand(), *d.values())


def test_gemm_gated_refusals():
    assert product(a=operand(rows=0)) == 0
    assert status_of(mx.mx_gemm_gated, operand(), operand(), None, 3, 0x40000, 128, None, 0, None, None) == INVALID
    for bad in (dict(act=-1), dict(act=4), dict(c=0), dict(ldc=127), dict(ld_preact=255), dict(up=operand(rows=127)),
                dict(up=operand(k=128)), dict(up=operand(orient=mx.MX_COLWISE)), dict(gate=operand(orient=mx.MX_COLWISE)),
                dict(a=operand(k=128)), dict(up=operand(data=0))):
        assert product(**bad) == INVALID, bad
    assert product(a=operand(k=48), gate=operand(k=48), up=operand(k=48)) == SHAPE
    assert product(gate=operand(rows=1 << 30), up=operand(rows=1 << 30), ldc=1 << 30, ld_preact=1 << 31) == SHAPE
    for bad in (dict(c=0x40001), dict(preact=0x50001), dict(up=operand(scale=0x20008)), dict(a=operand(data=0x10008))):
        assert product(**bad) == ALIGN, bad


def gate(back, **kw):
    d = dict(dh=0x1000, lddh=64) if back else {}
    d.update(gate_up=0x2000, ld=128, rows=32, f=64, act=mx.MX_ACT_SILU, axis=mx.MX_BOTH, **COPIES, group_offsets=None, n_groups=0,
             col_capacity=0, dev_status=None, stream=None)
    d.update(kw)
    return status_of(mx.mx_gated_backward_quantize if back else mx.mx_gated_quantize, *d.values())


@pytest.mark.parametrize("back", [False, True])
def test_gate_refusals(back):
    assert gate(back, rows=0) == 0
    assert gate(back, f=0) == 0
    groups = dict(group_offsets=0x9000, n_groups=4, col_capacity=512)
    for bad in (dict(rows=-1), dict(f=-32), dict(act=-1), dict(act=4), dict(axis=0), dict(axis=4), dict(gate_up=0), dict(ld=120),
                dict(row_data=None), dict(col_scale=None), {**groups, "n_groups": 0}, {**groups, "col_capacity": 500},
                {**groups, "col_capacity": -128}) + ((dict(dh=0), dict(lddh=56)) if back else ()):
        assert gate(back, **bad) == INVALID, bad
    for bad in (dict(f=48), dict(rows=40), dict(rows=1 << 31), {**groups, "n_groups": 513}):
        assert gate(back, **bad) == SHAPE, bad
    for bad in (dict(gate_up=0x2008), dict(ld=132), dict(row_scale=0x20008), {**groups, "group_offsets": 0x9004}) + (
            (dict(dh=0x1002), dict(lddh=68)) if back else ()):
        assert gate(back, **bad) == ALIGN, bad


def test_wrappers_refuse_before_the_library():
    """CPU tensors, wrong types and shapes: an assertion, not a pointer handed on."""
    x = torch.zeros(32, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, 64)
    for call in (lambda: mx.add_norm_quantize(f), lambda: mx.add_norm_quantize(x), lambda: mx.add_norm_quantize(x, x),
                 lambda: mx.add_norm_backward(x, x, None, f[:, 0]), lambda: mx.add_norm_backward(f, x, None, f[:, 0].contiguous()),
                 lambda: mx.gated_quantize(x), lambda: mx.gated_quantize(f), lambda: mx.gated_backward_quantize(x, x),
                 lambda: mx.gated_backward_quantize(x, torch.zeros(32, 128, dtype=torch.bfloat16))):
        with pytest.raises(AssertionError):
            call()
    t = mx.MXTensor(torch.zeros(32, 64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 32, 64, mx.MX_ROWWISE)
    with pytest.raises(AssertionError):
        mx.gemm_gated(t, t, t)
    with pytest.raises(KeyError):
        mx.gemm_gated(t, t, t, act="tanh")
