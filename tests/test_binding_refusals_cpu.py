"""The wrappers of the norms, the epilogue and the router take CUDA tensors only: a CPU
tensor's address must not reach a kernel. No GPU: the library's calls are stand-ins,
and a subclass passes for CUDA tensors."""
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx


class OnGpu(torch.Tensor):
    is_cuda = property(lambda self: True)


def cpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def gpu(*shape, dtype=torch.float32):
    return cpu(*shape, dtype=dtype).as_subclass(OnGpu)


def copy():
    return mx.MXTensor(gpu(64, 32, dtype=torch.uint8), gpu(512, dtype=torch.uint8), 64, 32, mx.MX_ROWWISE)


BF16, U8, I32 = torch.bfloat16, torch.uint8, torch.int32
X = (8, 16)

# every tensor of a call, as (shape, dtype)
CALLS = {
    "layer_norm": (lambda x, weight, bias, out: mx.layer_norm(x, weight, bias, out=out),
                   dict(x=(X, BF16), weight=((16,), torch.float32), bias=((16,), torch.float32), out=(X, BF16))),
    "layer_norm_backward": (lambda dy, x, weight, mean, rstd: mx.layer_norm_backward(dy, x, weight, mean, rstd),
                            dict(dy=(X, BF16), x=(X, BF16), weight=((16,), torch.float32), mean=((8,), torch.float32),
                                 rstd=((8,), torch.float32))),
    "gemm_epilogue": (lambda bias, residual, out, preact: mx.gemm_epilogue(mx.MX_FPROP, copy(), copy(), bias=bias, residual=residual,
                                                                           out=out, preact=preact),
                      dict(bias=((64,), BF16), residual=((64, 64), BF16), out=((64, 64), BF16), preact=((64, 64), BF16))),
    "epilogue_backward": (lambda dy, preact, dz: mx.epilogue_backward(dy, preact, "silu", dz=dz),
                          dict(dy=(X, BF16), preact=(X, BF16), dz=(X, BF16))),
    "router_forward": (lambda logits, token_mask: mx.router_forward(logits, 2, token_mask=token_mask),
                       dict(logits=(X, torch.float32), token_mask=((8,), U8))),
    "router_backward": (lambda logits, indices, load, dweights, dloss, token_mask:
                        mx.router_backward(logits, indices, load, dweights, dloss, token_mask=token_mask),
                        dict(logits=(X, torch.float32), indices=((8, 2), I32), load=((1, 16), torch.float32),
                             dweights=((8, 2), torch.float32), dloss=((1,), torch.float32), token_mask=((8,), U8))),
}


@pytest.fixture
def launches(monkeypatch):
    seen = []
    for name in mx.EXPORTED:
        if hasattr(mx, name) and not name.endswith("_bytes"):
            monkeypatch.setattr(mx, name, lambda *a, name=name: seen.append(name))
    monkeypatch.setattr(mx, "_stream", lambda s: None)
    return seen


@pytest.mark.parametrize("name", CALLS)
def test_cuda_tensors_are_taken(name, launches):
    call, args = CALLS[name]
    call(**{k: gpu(*shape, dtype=dtype) for k, (shape, dtype) in args.items()})
    assert len(launches) == 1


@pytest.mark.parametrize("name,which", [(n, a) for n, (_, args) in CALLS.items() for a in args])
def test_a_cpu_tensor_is_refused(name, which, launches):
    call, args = CALLS[name]
    with pytest.raises(AssertionError):
        call(**{k: (cpu if k == which else gpu)(*shape, dtype=dtype) for k, (shape, dtype) in args.items()})
    assert not launches
