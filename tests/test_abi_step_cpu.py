"""Host-side refusals of the operators around the products (no GPU needed):
every invalid argument is rejected before any device work."""
import os

import pytest

import mxfp8_block_scaled_gb300 as mx

INVALID, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module")
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


def adamw_tensor(**kw):
    d = dict(param=0x1000, grad=0x2000, exp_avg=0x3000, exp_avg_sq=0x4000, exp_avg_scale=0x5000, exp_avg_sq_scale=0x6000,
             numel=100, weight_decay=0.0, grad_dtype=mx.MX_F32, reserved=0)
    d.update(kw)
    return mx.MXAdamWTensorC(**d)


def adamw(tensor=None, bits=32, n=1, **hyper):
    h = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, seed=0, reserved=0)
    h.update(hyper)
    t = (mx.MXAdamWTensorC * 1)(tensor or adamw_tensor())
    return status_of(mx.mx_adamw_step, t, n, bits, mx.MXAdamWHyperC(**h), None, None, None)


def test_adamw_refusals(L):
    assert adamw(n=0) == 0
    assert adamw(n=-1) == INVALID
    assert adamw(bits=16) == INVALID
    for bad in (dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")),
                dict(eps=-1.0), dict(eps=float("inf")), dict(step=0), dict(reserved=1)):
        assert adamw(**bad) == INVALID, bad
    for bad in (dict(param=0), dict(grad=0), dict(exp_avg=0), dict(exp_avg_sq=0), dict(numel=-1), dict(grad_dtype=2),
                dict(reserved=1), dict(weight_decay=float("inf"))):
        assert adamw(adamw_tensor(**bad)) == INVALID, bad
    assert adamw(adamw_tensor(exp_avg_scale=0), bits=8) == INVALID
    for bad in (dict(param=0x1002), dict(grad=0x2002), dict(exp_avg=0x3001), dict(exp_avg_sq=0x4002)):
        assert adamw(adamw_tensor(**bad)) == ALIGN, bad
    assert adamw(adamw_tensor(grad=0x2001, grad_dtype=mx.MX_BF16)) == ALIGN
    assert adamw(adamw_tensor(exp_avg_scale=0x5002), bits=8) == ALIGN
    t = (mx.MXAdamWTensorC * 1)(adamw_tensor())
    h = mx.MXAdamWHyperC(1e-3, 0.9, 0.999, 1e-8, 1, 0, 0)
    assert status_of(mx.mx_adamw_step, None, 1, 32, h, None, None, None) == INVALID
    assert status_of(mx.mx_adamw_step, t, 1, 32, None, None, None, None) == INVALID
    assert status_of(mx.mx_adamw_step, t, 1, 32, h, 0x7002, None, None) == ALIGN


def norm(**kw):
    d = dict(x=0x1000, ldx=64, weight=0x2000, bias=0x3000, param_dtype=mx.MX_F32, rows=4, cols=64, eps=1e-5, center=1,
             dtype=mx.MX_BF16, y=0x4000, ldy=64, mean=0x5000, rstd=0x6000, dev_status=None, stream=None)
    d.update(kw)
    return status_of(mx.mx_layer_norm, *d.values())


def norm_backward(**kw):
    d = dict(dy=0x1000, lddy=64, x=0x2000, ldx=64, weight=0x3000, param_dtype=mx.MX_F32, mean=0x4000, rstd=0x5000, rows=4,
             cols=64, center=1, dtype=mx.MX_BF16, dx=0x6000, lddx=64, dweight=0x7000, dbias=0x8000, workspace=0x9000,
             workspace_bytes=1 << 20, dev_status=None, stream=None)
    d.update(kw)
    return status_of(mx.mx_layer_norm_backward, *d.values())


def test_norm_refusals(L):
    assert norm(rows=0) == 0
    for bad in (dict(rows=-1), dict(cols=0), dict(dtype=2), dict(param_dtype=-1), dict(center=2), dict(eps=-1.0),
                dict(eps=float("nan")), dict(x=0), dict(y=0), dict(ldx=63), dict(ldy=63)):
        assert norm(**bad) == INVALID, bad
    assert norm(cols=1 << 31, ldx=1 << 31, ldy=1 << 31) == SHAPE
    for bad in (dict(x=0x1001), dict(y=0x4001), dict(weight=0x2002), dict(bias=0x3001), dict(mean=0x5002), dict(rstd=0x6001),
                dict(x=0x1002, dtype=mx.MX_F32)):
        assert norm(**bad) == ALIGN, bad


def test_norm_backward_refusals(L):
    assert norm_backward(rows=0, dweight=None, dbias=None) == 0
    for bad in (dict(rows=-1), dict(cols=0), dict(dtype=2), dict(center=-1), dict(dy=0), dict(x=0), dict(dx=0), dict(mean=None),
                dict(rstd=None), dict(lddy=63), dict(lddx=63), dict(workspace=None), dict(workspace_bytes=100)):
        assert norm_backward(**bad) == INVALID, bad
    for bad in (dict(dx=0x6001), dict(workspace=0x9008), dict(dweight=0x7002), dict(rstd=0x5001)):
        assert norm_backward(**bad) == ALIGN, bad
    assert mx.mx_layer_norm_backward_workspace_bytes(4, 64) == 4 * 2 * 64 * 4
    assert mx.mx_layer_norm_backward_workspace_bytes(1 << 20, 64) == 304 * 2 * 64 * 4
    assert mx.mx_layer_norm_backward_workspace_bytes(0, 64) == 0


def operand(data=0x10000, scale=0x20000, rows=128, k=256, ld=0, orient=mx.MX_ROWWISE):
    return mx.MXOperandC(data, scale, rows, k, ld, orient, 0)


def epilogue(a=None, b=None, c=0x40000, ldc=128, mode=mx.MX_FPROP, **kw):
    d = dict(bias=0x1000, residual=0x2000, preact=0x3000, ld_residual=128, ld_preact=128, bias_dtype=mx.MX_F32,
             act=mx.MX_ACT_GELU)
    d.update(kw)
    return status_of(mx.mx_gemm_epilogue, mode, a or operand(), b or operand(), mx.MXEpilogueC(**d), c, ldc, None, None)


def test_epilogue_refusals(L):
    assert epilogue(a=operand(rows=0)) == 0
    for bad in (dict(act=-1), dict(act=4), dict(bias_dtype=2), dict(ld_residual=127), dict(ld_preact=127), dict(c=0),
                dict(ldc=127), dict(mode=mx.MX_DGRAD), dict(a=operand(k=128))):
        assert epilogue(**bad) == INVALID, bad
    assert status_of(mx.mx_gemm_epilogue, mx.MX_FPROP, operand(), operand(), None, 0x40000, 128, None, None) == INVALID
    assert epilogue(a=operand(k=48), b=operand(k=48)) == SHAPE
    for bad in (dict(bias=0x1002), dict(bias=0x1001, bias_dtype=mx.MX_BF16), dict(residual=0x2001), dict(preact=0x3001),
                dict(c=0x40001), dict(a=operand(data=0x10008))):
        assert epilogue(**bad) == ALIGN, bad


def epilogue_backward(**kw):
    d = dict(dy=0x1000, lddy=512, preact=0x2000, ld_preact=512, rows=64, cols=512, act=mx.MX_ACT_SILU, dz=0x3000, lddz=512,
             dbias=0x4000, workspace=0x5000, workspace_bytes=1 << 24, dev_status=None, stream=None)
    d.update(kw)
    return status_of(mx.mx_epilogue_backward, *d.values())


def test_epilogue_backward_refusals(L):
    assert epilogue_backward(cols=0) == 0
    assert epilogue_backward(dz=None, dbias=None) == 0
    assert epilogue_backward(rows=0, dbias=None) == 0
    for bad in (dict(rows=-1), dict(cols=-1), dict(act=4), dict(dy=0), dict(preact=None), dict(lddy=511), dict(ld_preact=511),
                dict(lddz=511), dict(workspace=None), dict(workspace_bytes=16)):
        assert epilogue_backward(**bad) == INVALID, bad
    assert epilogue_backward(rows=1 << 31) == SHAPE
    for bad in (dict(dy=0x1001), dict(preact=0x2001), dict(dz=0x3001), dict(dbias=0x4002), dict(workspace=0x5008)):
        assert epilogue_backward(**bad) == ALIGN, bad
    assert mx.mx_epilogue_backward_workspace_bytes(8, 512) == 0          # one CTA deep: straight into dbias
    assert mx.mx_epilogue_backward_workspace_bytes(64, 512) == 8 * 512 * 4
    assert mx.mx_epilogue_backward_workspace_bytes(0, 512) == 0


def router_forward(**kw):
    d = dict(logits=0x1000, ld=64, dtype=mx.MX_F32, token_mask=None, tokens=100, tokens_per_seq=50, n_experts=64, top_k=6,
             normalize=0, coef=1.0, indices=0x2000, weights=0x3000, counts=0x4000, group_offsets=0x5000, load=0x6000,
             loss=0x7000, workspace=0x8000, workspace_bytes=1 << 24, dev_status=None, stream=None)
    d.update(kw)
    return status_of(mx.mx_router_forward, *d.values())


def router_backward(**kw):
    d = dict(logits=0x1000, ld=64, dtype=mx.MX_F32, token_mask=None, tokens=100, tokens_per_seq=50, n_experts=64, top_k=6,
             normalize=0, indices=0x2000, load=0x3000, dweights=0x4000, dloss=0x5000, dlogits=0x6000, lddx=64,
             dev_status=None, stream=None)
    d.update(kw)
    return status_of(mx.mx_router_backward, *d.values())


def test_router_refusals(L):
    assert router_backward(tokens=0) == 0
    common = (dict(dtype=2), dict(tokens=-1), dict(tokens_per_seq=0), dict(n_experts=0), dict(top_k=0), dict(top_k=65),
              dict(normalize=2), dict(logits=0), dict(ld=63), dict(load=None))
    for bad in common + (dict(coef=float("nan")), dict(indices=None), dict(weights=None), dict(counts=None),
                         dict(group_offsets=None), dict(loss=None), dict(workspace=None), dict(workspace_bytes=64)):
        assert router_forward(**bad) == INVALID, bad
    for bad in common + (dict(indices=None), dict(dlogits=0), dict(lddx=63)):
        assert router_backward(**bad) == INVALID, bad
    for bad in (dict(n_experts=513, ld=513), dict(tokens=1 << 31)):
        assert router_forward(**bad) == SHAPE and router_backward(**bad, lddx=513) == SHAPE, bad
    for bad in (dict(logits=0x1002), dict(counts=0x4004), dict(group_offsets=0x5004), dict(weights=0x3002), dict(loss=0x7001),
                dict(workspace=0x8008), dict(load=0x6002), dict(indices=0x2001)):
        assert router_forward(**bad) == ALIGN, bad
    for bad in (dict(dlogits=0x6002), dict(dweights=0x4001), dict(dloss=0x5002), dict(load=0x3001), dict(indices=0x2002)):
        assert router_backward(**bad) == ALIGN, bad
    assert mx.mx_router_workspace_bytes(0, 1, 64) == 0
    # 4 CTAs of 32 tokens (two sequences of 50): (4 + 2) rows of 64 x 8 bytes, and the counts of valid tokens
    assert mx.mx_router_workspace_bytes(100, 50, 64) == 6 * 64 * 8 + 16 + 16
