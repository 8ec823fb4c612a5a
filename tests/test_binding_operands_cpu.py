"""The products' wrappers take operands of CUDA tensors only: a CPU tensor's address must
not reach a kernel, whichever of an operand's two tensors it is; and outputs, workspaces
and group offsets on the GPU, as the quantisers take theirs, and every call its status
word. No GPU: the library's calls are stand-ins."""
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


def blockwise(block, make_data=gpu, make_scale=gpu):
    return mx.FP8Blockwise(make_data(128, 128, dtype=U8), make_scale(1, 128), 128, 128, block)


def copies(make):
    row = mx.MXTensor(make(64, 32, dtype=U8), make(512, dtype=U8), 64, 32, mx.MX_ROWWISE)
    return row, mx.MXTensor(make(32, 128, dtype=U8), make(512, dtype=U8), 32, 128, mx.MX_COLWISE)


a, b, s = operand(), operand(), stacked()
OTHERS = {   # every other tensor of a product's call, made here by `make`
    "gemm out": lambda make: mx.gemm(mx.MX_FPROP, a, b, out=make(*OUT, dtype=BF16)),
    "gemm_with_workspace out": lambda make: mx.gemm(mx.MX_FPROP, a, b, out=make(*OUT, dtype=BF16), workspace=gpu(512, dtype=U8)),
    "gemm_with_workspace workspace": lambda make: mx.gemm(mx.MX_FPROP, a, b, out=gpu(*OUT, dtype=BF16), workspace=make(512, dtype=U8)),
    "gemm_multi out": lambda make: mx.gemm_multi([(mx.MX_FPROP, a, b, make(*OUT, dtype=BF16))]),
    "gemm_gated out": lambda make: mx.gemm_gated(a, b, b, out=make(*OUT, dtype=BF16)),
    "gemm_current out": lambda make: mx.gemm_current(mx.MX_FPROP, a, b, out=make(*OUT, dtype=BF16)),
    "gemm_current_multi out": lambda make: mx.gemm_current_multi([(mx.MX_FPROP, a, b, make(*OUT, dtype=BF16))]),
    "grouped_gemm out": lambda make: mx.grouped_gemm(mx.MX_FPROP, a, s, gpu(3, dtype=I64), out=make(*OUT, dtype=BF16)),
    "grouped_gemm offsets": lambda make: mx.grouped_gemm(mx.MX_FPROP, a, s, make(3, dtype=I64), out=gpu(*OUT, dtype=BF16)),
    "grouped_gemm_current out": lambda make: mx.grouped_gemm_current(mx.MX_FPROP, a, s, gpu(3, dtype=I64), out=make(*OUT, dtype=BF16)),
    "grouped_gemm_current offsets": lambda make: mx.grouped_gemm_current(mx.MX_FPROP, a, s, make(3, dtype=I64), out=gpu(*OUT, dtype=BF16)),
    "grouped_gemm_swiglu out": lambda make: mx.grouped_gemm_swiglu(a, s, gpu(3, dtype=I64), out=make(64, 32, dtype=BF16)),
    "grouped_gemm_swiglu offsets": lambda make: mx.grouped_gemm_swiglu(a, s, make(3, dtype=I64), out=gpu(64, 32, dtype=BF16)),
    "grouped_gemm_swiglu_quantize out": lambda make: mx.grouped_gemm_swiglu_quantize(a, s, gpu(3, dtype=I64), 128, out=copies(make)),
    "grouped_gemm_swiglu_quantize offsets": lambda make: mx.grouped_gemm_swiglu_quantize(a, s, make(3, dtype=I64), 128, out=copies(gpu)),
    "gemm_fp8_blockwise out": lambda make: mx.gemm_fp8_blockwise(blockwise(1), blockwise(128), out=make(128, 128, dtype=BF16)),
    "gemm_fp8_blockwise a": lambda make: mx.gemm_fp8_blockwise(blockwise(1, make), blockwise(128), out=gpu(128, 128, dtype=BF16)),
    "gemm_fp8_blockwise b": lambda make: mx.gemm_fp8_blockwise(blockwise(1), blockwise(128, gpu, make), out=gpu(128, 128, dtype=BF16)),
}
X = (64, 32)
OTHERS.update({   # the quantisers'
    "quantize offsets": lambda make: mx.quantize(gpu(*X, dtype=BF16), mx.MX_BOTH, group_offsets=make(3, dtype=I64)),
    "quantize status": lambda make: mx.quantize(gpu(*X, dtype=BF16), status=make(1, dtype=torch.int32)),
    "quantize_batched w": lambda make: mx.quantize_stacked(make(2, *X, dtype=BF16), mx.MX_BOTH),
    "quantize_f32 w": lambda make: mx.quantize_stacked(make(2, *X), mx.MX_BOTH),
    "quantize_current x": lambda make: mx.quantize_current(make(*X, dtype=BF16), amax=gpu(1)),
    "quantize_current amax": lambda make: mx.quantize_current(gpu(*X, dtype=BF16), amax=make(1)),
    "quantize_current offsets": lambda make: mx.quantize_current(gpu(*X, dtype=BF16), amax=gpu(1), group_offsets=make(3, dtype=I64)),
    "gated_quantize offsets": lambda make: mx.gated_quantize(gpu(64, 64, dtype=BF16), group_offsets=make(3, dtype=I64)),
    "gated_quantize status": lambda make: mx.gated_quantize(gpu(64, 64, dtype=BF16), status=make(1, dtype=torch.int32)),
    "add_norm_quantize status": lambda make: mx.add_norm_quantize(gpu(*X, dtype=BF16), status=make(1, dtype=torch.int32)),
    "gemm status": lambda make: mx.gemm(mx.MX_FPROP, a, b, out=gpu(*OUT, dtype=BF16), status=make(1, dtype=torch.int32)),
})


@pytest.mark.parametrize("name", OTHERS)
def test_other_tensors_on_the_cpu_are_refused(name, launches):  # noqa: F811
    OTHERS[name](gpu)
    assert launches == ["mx_" + name.split()[0]]
    with pytest.raises(AssertionError):
        OTHERS[name](cpu)
    assert len(launches) == 1
