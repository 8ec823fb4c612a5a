"""A wait inside the norms that runs out shows in the results, with a status word or
without: a stage that waits for bytes nothing sends gives up after its limit, its rows
and the gradients they are part of are NaN (but for a first or last row that is read
without copies, which is right), and the context stays usable. (The refusals
of the self test need no GPU: tests/test_abi_norm_timeout_cpu.py.)"""
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import workloads

pytestmark = pytest.mark.gpu
LIMIT = 2_000_000     # ns


def lost_rows(got, right):
    """Which rows are NaN throughout; the others are right, and the first or the last
    row of rows off the 16-byte boundaries."""
    rows, cols = got.shape
    nan = torch.isnan(got)
    lost = nan.all(1)
    assert torch.equal(nan.any(1), lost) and torch.equal(got[~lost], right[~lost])
    kept = set((~lost).nonzero().flatten().tolist())
    assert kept <= ({0, rows - 1} if cols * 2 % 16 else set()), kept
    return lost


SHAPES = [(1, 257), (5, 264), (700, 513), (3, 1024), (5000, 2048), (9, 2047), (400, 7168), (4, 8191), (2, 16384), (3, 12001)]


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("with_status", [True, False])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, with_status):
    x = workloads.normal_bf16((rows, cols), 1).cuda()
    out, rstd = torch.zeros_like(x), torch.zeros(rows, device="cuda")
    st = mx.new_status()
    mx.mx_selftest_norm_timeout(LIMIT, None, x.data_ptr(), rows, cols, out.data_ptr(), rstd.data_ptr(), None, None, None, 0,
                                st.data_ptr() if with_status else None, stream())
    torch.cuda.synchronize()
    assert mx.STATUS_NAMES[mx.read_status(st)] == ("MX_ERR_TIMEOUT" if with_status else "MX_OK")
    st.zero_()
    y, _, r = mx.layer_norm(x, center=False, status=st)          # the next call is not touched by it
    assert mx.read_status(st) == 0 and torch.isfinite(y).all() and torch.isfinite(r).all()
    lost = lost_rows(out, y)
    assert torch.isnan(rstd[lost]).all() and torch.equal(rstd[~lost], r[~lost])


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(rows, cols):
    x, dy = (workloads.normal_bf16((rows, cols), i).cuda() for i in (1, 2))
    rstd = torch.ones(rows, device="cuda")
    out, dw, db = torch.zeros_like(x), torch.zeros(cols, device="cuda"), torch.zeros(cols, device="cuda")
    need = mx.mx_layer_norm_backward_workspace_bytes(rows, cols)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    st = mx.new_status()
    mx.mx_selftest_norm_timeout(LIMIT, dy.data_ptr(), x.data_ptr(), rows, cols, out.data_ptr(), rstd.data_ptr(), dw.data_ptr(),
                                db.data_ptr(), ws.data_ptr(), need, st.data_ptr(), stream())
    torch.cuda.synchronize()
    assert mx.STATUS_NAMES[mx.read_status(st)] == "MX_ERR_TIMEOUT"
    st.zero_()
    got = mx.layer_norm_backward(dy, x, None, None, rstd, center=False, status=st)
    assert mx.read_status(st) == 0 and all(torch.isfinite(t).all() for t in got)
    if lost_rows(out, got[0]).any():
        assert torch.isnan(dw).all() and torch.isnan(db).all()
    else:
        assert torch.equal(dw, got[1]) and torch.equal(db, got[2])
