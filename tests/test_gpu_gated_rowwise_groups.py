"""The gate's row copies alone, with the experts' offsets given: the copies of the dense
call, byte for byte, and the offsets are not read (a row copy has no segments), so that
ones for other rows are no error."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
from tests.test_gpu_gated import check_gate, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,F", [([100, 0, 156], 96), ([37, 0, 300, 1, 128], 352), ([1], 32), ([5, 127, 128, 0, 0, 1000, 33, 2], 1408)])
def test_row_copies_do_not_depend_on_groups(counts, F):
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    M = int(offs[-1])
    z, dh = normal(M, 2 * F, 25, 2.0), normal(M, F, 26, 0.1)
    right, wrong = (torch.from_numpy(o).cuda() for o in (offs, offs + 7))
    dense = mx.gated_quantize(z, axis=mx.MX_ROWWISE)[0], mx.gated_backward_quantize(dh, z, axis=mx.MX_ROWWISE)[0]
    check_gate(z, dh, "silu", dense[0], None, dense[1], None)
    for o in (right, wrong):
        st = mx.new_status()
        kw = dict(axis=mx.MX_ROWWISE, group_offsets=o, col_capacity=mx.mx_grouped_padded_rows(offs), status=st)
        got = mx.gated_quantize(z, **kw), mx.gated_backward_quantize(dh, z, **kw)
        assert mx.read_status(st) == 0
        for (row, col), want in zip(got, dense):
            assert col is None and torch.equal(row.data, want.data) and torch.equal(row.scale, want.scale)
