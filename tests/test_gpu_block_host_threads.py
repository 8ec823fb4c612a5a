"""The gated block's calls from several host threads at once, each on its own stream with
its own sizes (kernels shared, splits and shared memory not), while another thread's next
launch was asked to run out of time: that one alone does."""
import threading

import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import workloads

pytestmark = pytest.mark.gpu
CALLS = 400
BF16 = torch.bfloat16


def normal(rows, cols, seed):
    return workloads.normal_bf16((rows, cols), seed).cuda()


def norms(cols):
    x, res, dy, w = normal(96, cols, 1), normal(96, cols, 2), normal(96, cols, 3), torch.ones(cols, device="cuda")

    def call(stream):
        n = mx.add_norm_quantize(x, res, w, stream=stream)
        b = mx.add_norm_backward(dy, n.sum, w, n.rstd, dsum=res, axis=mx.MX_BOTH, stream=stream)
        return [n.sum, n.rstd, n.row.data, n.col.data, n.col.scale, b.dx, b.dweight, b.row.data, b.col.data]

    return call


def gates(F):
    z, dh = normal(160, 2 * F, 4), normal(160, F, 5)

    def call(stream):
        return [t for c in (*mx.gated_quantize(z, stream=stream), *mx.gated_backward_quantize(dh, z, stream=stream))
                for t in (c.data, c.scale)]

    return call


def product(M):
    a, g, u = (mx.quantize(normal(r, 512, r + i), mx.MX_ROWWISE)[0] for i, r in enumerate((M, 352, 352)))
    return lambda stream: [t for t in mx.gemm_gated(a, g, u, keep_preact=True, stream=stream)]


@pytest.mark.parametrize("make,sizes", [(norms, (2048, 8192, 544)), (gates, (96, 1408)), (product, (1, 20, 300))])
def test_threads(make, sizes):
    calls = [make(n) for n in sizes]
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    mx.mx_selftest_block_timeout(1, 2_000_000)      # this thread's next launch, which the others do not make
    wrong = []

    def run(call, right):
        try:
            stream = torch.cuda.Stream()
            for i in range(CALLS):
                got = call(stream)
                if i % 50 == 0:
                    stream.synchronize()
                    if not all(torch.equal(p, q) for p, q in zip(got, right)):
                        wrong.append(i)
        except Exception as e:      # a thread's failure is the test's
            wrong.append(repr(e))

    threads = [threading.Thread(target=run, args=x) for x in zip(calls, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    mx.mx_selftest_block_timeout(0, 0)
    assert not wrong, wrong
    for c, w in zip(calls, want):
        assert all(torch.equal(p, q) for p, q in zip(c(None), w))
