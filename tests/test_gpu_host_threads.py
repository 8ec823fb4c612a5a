"""Calls from several host threads at once, each thread on its own stream with its
own sizes: norms whose widths share a kernel but not its shared memory."""
import threading

import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import workloads

pytestmark = pytest.mark.gpu
CALLS = 15000


def forward(cols):
    x = workloads.normal_bf16((2, cols), cols).cuda()
    y = torch.empty_like(x)
    want = mx.layer_norm(x)[0]
    def call(stream):
        mx.mx_layer_norm(x.data_ptr(), cols, None, None, mx.MX_F32, 2, cols, 1e-5, 1, mx.MX_BF16, y.data_ptr(), cols, None, None,
                         None, stream)
    return call, lambda: torch.equal(y, want)


def backward(cols):
    x, dy = (workloads.normal_bf16((2, cols), cols + i).cuda() for i in range(2))
    _, mean, rstd = mx.layer_norm(x)
    dx = torch.empty_like(x)
    want = mx.layer_norm_backward(dy, x, None, mean, rstd)[0]
    def call(stream):
        mx.mx_layer_norm_backward(dy.data_ptr(), cols, x.data_ptr(), cols, None, mx.MX_F32, mean.data_ptr(), rstd.data_ptr(), 2,
                                  cols, 1, mx.MX_BF16, dx.data_ptr(), cols, None, None, None, 0, None, stream)
    return call, lambda: torch.equal(dx, want)


@pytest.mark.parametrize("make,widths", [(forward, (8192, 4104)), (forward, (16384, 8200)), (backward, (8192, 4104)),
                                         (backward, (16384, 8200))])
def test_norms_of_two_widths(make, widths):
    work = [make(c) for c in widths]
    streams = [torch.cuda.Stream() for _ in widths]
    torch.cuda.synchronize()
    failed = []
    def run(call, stream):
        try:
            for _ in range(CALLS):
                call(stream.cuda_stream)
        except mx.MXError as e:
            failed.append(str(e))
    threads = [threading.Thread(target=run, args=(call, s)) for (call, _), s in zip(work, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert all(right() for _, right in work)
