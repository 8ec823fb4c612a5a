"""The products' wrappers take operands of CUDA tensors only: a CPU tensor's address must
not reach a kernel, whichever of an operand's two tensors it is. No GPU: the library's
calls are stand-ins."""
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
from tests.test_binding_refusals_cpu import cpu, gpu, launches  # noqa: F401 (a fixture)

BF16, U8, I64 = torch.bfloat16, torch.uint8, torch.int64


def operand(make_data=gpu, make_scale=gpu):
    return mx.MXTensor(make_data(64, 32, dtype=U8), make_scale(512, dtype=U8), 64, 32, mx.MX_ROWWISE)


def stacked(make_data=gpu, make_scale=gpu):
    return mx.MXStacked(make_data(2, 64, 32, dtype=U8), make_scale(2, 512, dtype=U8), 64, 32, mx.MX_ROWWISE)


OUT = (64, 64)
CALLS = {   # the call, and how its operands are made
    "gemm_gated": (lambda a, b, c: mx.gemm_gated(a, b, c, out=gpu(*OUT, dtype=BF16)), (operand, operand, operand)),
    "gemm": (lambda a, b: mx.gemm(mx.MX_FPROP, a, b, out=gpu(*OUT, dtype=BF16)), (operand, operand)),
    "gemm_multi": (lambda a, b: mx.gemm_multi([(mx.MX_FPROP, a, b, gpu(*OUT, dtype=BF16))]), (operand, operand)),
    "gemm_epilogue": (lambda a, b: mx.gemm_epilogue(mx.MX_FPROP, a, b, out=gpu(*OUT, dtype=BF16)), (operand, operand)),
    "gemm_current": (lambda a, b: mx.gemm_current(mx.MX_FPROP, a, b, out=gpu(*OUT, dtype=BF16)), (operand, operand)),
    "grouped_gemm": (lambda a, b: mx.grouped_gemm(mx.MX_FPROP, a, b, gpu(3, dtype=I64), out=gpu(*OUT, dtype=BF16)),
                     (operand, stacked)),
    "grouped_gemm_swiglu": (lambda a, b: mx.grouped_gemm_swiglu(a, b, gpu(3, dtype=I64), out=gpu(64, 32, dtype=BF16)),
                            (operand, stacked)),
}


@pytest.mark.parametrize("name", CALLS)
def test_operands_on_the_gpu_are_taken(name, launches):  # noqa: F811
    call, makers = CALLS[name]
    call(*[make() for make in makers])
    assert launches == ["mx_" + name]


@pytest.mark.parametrize("part", [0, 1])
@pytest.mark.parametrize("name,which", [(n, i) for n, (_, makers) in CALLS.items() for i in range(len(makers))])
def test_an_operand_on_the_cpu_is_refused(name, which, part, launches):  # noqa: F811
    call, makers = CALLS[name]
    tensors = [cpu if part == 0 else gpu, cpu if part == 1 else gpu]
    with pytest.raises(AssertionError):
        call(*[make(*tensors) if i == which else make() for i, make in enumerate(makers)])
    assert not launches
