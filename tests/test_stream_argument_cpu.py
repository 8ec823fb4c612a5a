"""What a wrapper allocates belongs to the stream it is given (no GPU: the library
calls and torch's streams are stand-ins that record what happens under which)."""
import contextlib

import pytest
import torch

import mxfp8_block_scaled_gb300 as mx


class OnGpu(torch.Tensor):
    """A CPU tensor that passes for a CUDA one in the wrappers' checks."""
    is_cuda = property(lambda self: True)


def tensor(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


class Side:
    cuda_stream = 0x5EED


def copy(rows, k, orient=mx.MX_ROWWISE):
    return mx.MXTensor(tensor(rows, k, dtype=torch.uint8), tensor(512, dtype=torch.uint8), rows, k, orient)


def stacked(n, rows, k):
    return mx.MXStacked(tensor(n, rows, k, dtype=torch.uint8), tensor(n, 512, dtype=torch.uint8), rows, k, mx.MX_ROWWISE)


BF16, I32, I64 = torch.bfloat16, torch.int32, torch.int64
x, logits, offsets = tensor(600, 64, dtype=BF16), tensor(600, 8), tensor(3, dtype=I64)
stat = tensor(600)


def blockwise(block):
    return mx.FP8Blockwise(tensor(128, 128, dtype=torch.uint8), tensor(128, 1), 128, 128, block)


CALLS = {
    "layer_norm": lambda s: mx.layer_norm(x, stream=s),
    "layer_norm_backward": lambda s: mx.layer_norm_backward(x, x, None, stat, stat, stream=s),
    "gemm_epilogue": lambda s: mx.gemm_epilogue(mx.MX_FPROP, copy(64, 32), copy(96, 32), keep_preact=True, stream=s),
    "epilogue_backward": lambda s: mx.epilogue_backward(x, x, "gelu", stream=s),
    "router_forward": lambda s: mx.router_forward(logits, 2, stream=s),
    "router_backward": lambda s: mx.router_backward(logits, tensor(600, 2, dtype=I32), tensor(1, 8), stream=s),
    "quantize": lambda s: mx.quantize(x, stream=s),
    "quantize_multi": lambda s: mx.quantize_multi([x, x], stream=s),
    "quantize_stacked": lambda s: mx.quantize_stacked(tensor(2, 64, 32, dtype=BF16), mx.MX_BOTH, stream=s),
    "quantize_current": lambda s: mx.quantize_current(x, stream=s),       # its amax is dropped on return
    "current_amax": lambda s: mx.current_amax(x, stream=s),
    "gemm": lambda s: mx.gemm(mx.MX_FPROP, copy(64, 32), copy(96, 32), None, None, s),    # by position
    "gemm_multi": lambda s: mx.gemm_multi([(mx.MX_FPROP, copy(64, 32), copy(96, 32))], stream=s),
    "gemm_current": lambda s: mx.gemm_current(mx.MX_FPROP, copy(64, 32), copy(96, 32), stream=s),
    "gemm_current_multi": lambda s: mx.gemm_current_multi([(mx.MX_FPROP, copy(64, 32), copy(96, 32))], stream=s),
    "grouped_gemm": lambda s: mx.grouped_gemm(mx.MX_FPROP, copy(64, 32), stacked(2, 96, 32), offsets, stream=s),
    "grouped_gemm_current": lambda s: mx.grouped_gemm_current(mx.MX_FPROP, copy(64, 32), stacked(2, 96, 32), offsets, stream=s),
    "grouped_gemm_swiglu": lambda s: mx.grouped_gemm_swiglu(copy(64, 32), stacked(2, 96, 32), offsets, stream=s),
    "grouped_gemm_swiglu_quantize": lambda s: mx.grouped_gemm_swiglu_quantize(copy(64, 32), stacked(2, 96, 32), offsets, 384,
                                                                              stream=s),
    "quantize_fp8_blockwise": lambda s: mx.quantize_fp8_blockwise(x, 1, stream=s),
    "gemm_fp8_blockwise": lambda s: mx.gemm_fp8_blockwise(blockwise(1), blockwise(128), stream=s),
}


@pytest.fixture
def record(monkeypatch):
    """(what, stream): every allocation and every library call, in order."""
    seen, under = [], [None]

    @contextlib.contextmanager
    def stream(handle):
        under.append(handle)
        yield
        under.pop()

    real = torch.empty

    def empty(*a, **k):
        seen.append(("empty", under[-1]))
        return real(*a, **k).as_subclass(OnGpu)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch, "empty", empty)
    for name in mx.EXPORTED:
        if hasattr(mx, name) and not name.endswith("_bytes"):
            monkeypatch.setattr(mx, name, lambda *a, name=name: seen.append((name, a[-1])))
    monkeypatch.setattr(mx, "_stream", lambda s: under[-1] if s is None else s.cuda_stream)
    return seen


@pytest.mark.parametrize("name", CALLS)
def test_allocations_belong_to_the_given_stream(name, record):
    CALLS[name](Side())
    assert any(what == "empty" for what, _ in record) and any(what != "empty" for what, _ in record)
    assert all(s == Side.cuda_stream for _, s in record), record


@pytest.mark.parametrize("name", CALLS)
def test_without_one_they_belong_to_the_current_stream(name, record):
    CALLS[name](None)
    assert record and all(s is None for _, s in record), record


def test_every_wrapper_with_a_stream_that_allocates_is_covered():
    import inspect
    have = {n for n, f in vars(mx).items() if inspect.isfunction(f) and not n.startswith(("_", "mx_"))
            and inspect.signature(f).parameters.get("stream")}
    assert have - set(CALLS) == {"adamw_step"}        # updates what it is given
