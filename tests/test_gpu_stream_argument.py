"""The wrappers' ``stream=`` argument: their scratch and outputs belong to that
stream. The side stream is kept busy with products, so the call's kernels run well
after it has returned, while the current stream's next allocations of the same
sizes are filled with other values."""
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import workloads

pytestmark = pytest.mark.gpu


def matrix(rows, cols, seed, dtype=torch.bfloat16):
    return workloads.normal_bf16((rows, cols), seed).cuda().to(dtype)


def norm_backward():
    x, dy = matrix(2000, 1024, 1), matrix(2000, 1024, 2)
    _, mean, rstd = mx.layer_norm(x)
    return (lambda **k: mx.layer_norm_backward(dy, x, None, mean, rstd, **k),
            mx.mx_layer_norm_backward_workspace_bytes(2000, 1024))


def epilogue_backward():
    dy, z = matrix(3000, 1024, 3), matrix(3000, 1024, 4)
    return (lambda **k: mx.epilogue_backward(dy, z, "gelu", **k), mx.mx_epilogue_backward_workspace_bytes(3000, 1024))


def router_forward():
    x = matrix(8192, 64, 5, torch.float32)
    def call(**k):
        r = mx.router_forward(x, 6, tokens_per_seq=1024, normalize=True, **k)
        return r.indices, r.weights, r.counts, r.group_offsets, r.load, r.loss
    return call, mx.mx_router_workspace_bytes(8192, 1024, 64)


def quantize_current():
    x = matrix(1024, 512, 6)
    def call(**k):
        row, col = mx.quantize_current(x, **k)
        return row.data, row.scale, col.data
    return call, 4


@pytest.mark.parametrize("make", [norm_backward, epilogue_backward, router_forward, quantize_current])
def test_scratch_is_not_handed_to_the_current_stream(make):
    call, scratch = make()
    want = [t.clone() for t in call()]
    a = matrix(4096, 4096, 7)
    b = torch.empty_like(a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(20):
                torch.matmul(a, a, out=b)
        got = call(stream=side)
        taken = [torch.full((max(scratch // 4, 1),), float("nan"), device="cuda") for _ in range(8)]
        taken += [torch.full_like(t, 77) for t in want for _ in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert all(torch.isnan(t).all() for t in taken[:8]) and all((t == 77).all() for t in taken[8:])


def test_the_next_kernels_of_the_current_stream_follow_by_an_event():
    x = matrix(300, 512, 8)
    want = mx.layer_norm(x)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = mx.layer_norm(x, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
