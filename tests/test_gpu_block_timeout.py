"""A wait that runs out inside the norms with the residual's addition, the gate or the
product of few tokens: MX_ERR_TIMEOUT where a status word is given, NaN in what the
wait was for and nowhere else, the context usable and the next call right. (The
refusals of the self test need no GPU: tests/test_abi_block_timeout_cpu.py.)"""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_gb300 as mx
import oracle
import workloads
from tests.gpu_util import u8

pytestmark = pytest.mark.gpu
LIMIT = 2_000_000     # ns
STAGES, SUMS = 1, 2
BF16, F32 = torch.bfloat16, torch.float32


def normal(shape, seed, std=1.0, dtype=BF16):
    return torch.from_numpy((workloads.philox(seed).standard_normal(shape) * std).astype(np.float32)).cuda().to(dtype)


def ran_out(call, what, with_status=True):
    """The call's outputs with a wait that runs out, and the same call's right ones from before and after it."""
    right = call(None)
    st = mx.new_status()
    mx.mx_selftest_block_timeout(what, LIMIT)
    got = call(st if with_status else None)
    torch.cuda.synchronize()
    assert mx.STATUS_NAMES[mx.read_status(st)] == ("MX_ERR_TIMEOUT" if with_status else "MX_OK")
    st.zero_()
    again = call(st)
    assert mx.read_status(st) == 0
    for a, b in zip(right, again):
        for p, q in zip(parts(a), parts(b)):
            assert torch.equal(p, q)
    return got, right


def parts(x):
    return [] if x is None else [x.data, x.scale] if isinstance(x, mx.MXTensor) else [x]


def check_lost(copy, right, lost):
    """A copy's blocks: codes 0x7F under scale 0xFF where `lost` (logical [rows, k/32]) says so, right elsewhere."""
    scales, want = (oracle.mx_scale_unswizzle(u8(c.scale), c.rows, c.k // 32) for c in (copy, right))
    assert np.array_equal(oracle.mx_scale_swizzle(scales), u8(copy.scale)), "scale padding"
    assert np.array_equal(scales, np.where(lost, 0xFF, want))
    codes, want = u8(copy.data), u8(right.data)
    wide = lost.repeat(32, 1)
    assert ((codes & 0x7F) == 0x7F)[wide].all() and np.array_equal(codes[~wide], want[~wide])


def all_lost(copy):
    return np.ones((copy.rows, copy.k // 32), dtype=bool)


# one warp, several, clusters of several sizes, rounds of panels, values held over the exchange and read again
SHAPES = [(1, 64, BF16), (96, 64, BF16), (33, 608, F32), (160, 2048, BF16), (64, 8192, BF16), (96, 8192, F32), (64, 16384, BF16), (64, 16384, F32),
          (12832, 2048, BF16), (6400, 2048, F32), (1056, 7168, F32), (2080, 10240, BF16)]


def norm_inputs(rows, cols, dtype):
    x, res = normal((rows, cols), 1, 0.5), normal((rows, cols), 2, 2.0, dtype)
    dy, ds = normal((rows, cols), 3, 0.1), normal((rows, cols), 4, 0.3, dtype)
    return x, res, dy, ds, 1.0 + normal((cols,), 5, 0.2, F32)


@pytest.mark.parametrize("with_status", [True, False])
@pytest.mark.parametrize("rows,cols,dtype", SHAPES)
def test_norm_stages(rows, cols, dtype, with_status):
    """Every stage: everything is NaN."""
    x, res, dy, ds, w = norm_inputs(rows, cols, dtype)
    axis = mx.MX_BOTH if rows % 32 == 0 else mx.MX_ROWWISE

    def forward(status):
        n = mx.add_norm_quantize(x, res, w, axis=axis, keep_output=True, status=status)
        return [n.row, n.col, n.sum, n.rstd, n.y]

    got, right = ran_out(forward, STAGES, with_status)
    assert all(torch.isnan(t).all() for t in got[2:])
    for c, r in zip(got[:2], right[:2]):
        if c is not None:
            check_lost(c, r, all_lost(c))
    total, rstd = right[2], right[3]

    def backward(status):
        b = mx.add_norm_backward(dy, total, w, rstd, dsum=ds, axis=axis, status=status)
        return [b.row, b.col, b.dx, b.dweight]

    got, right = ran_out(backward, STAGES, with_status)
    assert torch.isnan(got[2]).all() and torch.isnan(got[3]).all()
    for c, r in zip(got[:2], right[:2]):
        if c is not None:
            check_lost(c, r, all_lost(c))


def lost_panels(nan, rows, cols):
    """Of values [rows, cols] whose NaN are given: panels of 32 rows lost from one column on (the
    last CTA's), the same for all that are not lost throughout. Returns that mask by panel and block of 32 columns."""
    panels = nan.reshape(rows // 32, 32, cols)
    assert (panels == panels[:, :1]).all()                    # all rows of a panel alike
    first = panels[:, 0]
    start = np.where(first.any(1), first.argmax(1), cols)
    assert np.array_equal(first, np.arange(cols)[None] >= start[:, None])
    some = start[start > 0]
    assert len(some) == 0 or (some == some[0]).all() and some[0] % 64 == 0
    lost = start == 0
    # a cluster's first panel comes before its others: those lost throughout are the later ones
    assert (np.diff(lost.astype(int)) >= 0).all()
    return first[:, ::32]


@pytest.mark.parametrize("rows,cols,dtype", [s for s in SHAPES if s[0] % 32 == 0])
def test_norm_sums(rows, cols, dtype):
    """The last CTA of each cluster gets no rows' sums of its first panel and sends none from then on."""
    x, res, dy, ds, w = norm_inputs(rows, cols, dtype)

    def forward(status):
        n = mx.add_norm_quantize(x, res, w, keep_output=True, status=status)
        return [n.row, n.col, n.sum, n.rstd, n.y]

    def backward(status):
        b = mx.add_norm_backward(dy, total, w, rstd, dsum=ds, axis=mx.MX_BOTH, status=status)
        return [b.row, b.col, b.dx, b.dweight]

    def check(value, want, row, row_want, col, col_want):
        nan = torch.isnan(value).cpu().numpy()
        blocks = lost_panels(nan, rows, cols)
        keep = ~torch.from_numpy(nan).cuda()
        assert torch.equal(value[keep], want[keep])
        check_lost(row, row_want, blocks.repeat(32, 0))
        check_lost(col, col_want, blocks.T.repeat(32, 0))
        assert blocks.any()
        return blocks

    got, right = ran_out(forward, SUMS)
    total, rstd = right[2], right[3]
    assert torch.equal(got[2], right[2])
    blocks = check(got[4], right[4], got[0], right[0], got[1], right[1])
    lost = torch.from_numpy(blocks[:, 0].repeat(32)).cuda()      # the first CTA writes the statistic
    assert torch.isnan(got[3][lost]).all() and torch.equal(got[3][~lost], right[3][~lost])
    got, right = ran_out(backward, SUMS)
    assert torch.equal(got[3], right[3])
    check(got[2], right[2], got[0], right[0], got[1], right[1])


def test_norm_sums_lose_part_of_a_row():
    """More than one CTA a cluster: the first panel's other columns are right."""
    x, res, dy, ds, w = norm_inputs(64, 8192, BF16)
    call = lambda s: [mx.add_norm_quantize(x, res, w, keep_output=True, status=s).y]  # noqa: E731
    got, _ = ran_out(call, SUMS)
    nan = torch.isnan(got[0])
    assert nan.any() and not nan[:, 0].any()


@pytest.mark.parametrize("with_status", [True, False])
@pytest.mark.parametrize("rows,F", [(32, 32), (160, 352), (8192, 1408)])
def test_gate(rows, F, with_status):
    z, dh = normal((rows, 2 * F), 6), normal((rows, F), 7, 0.1)
    for call in (lambda s: mx.gated_quantize(z, status=s), lambda s: mx.gated_backward_quantize(dh, z, status=s)):
        got, right = ran_out(call, STAGES, with_status)
        for c, r in zip(got, right):
            check_lost(c, r, all_lost(c))


@pytest.mark.parametrize("rows", [1, 33, 500])
def test_gate_row_copies(rows):
    z, dh = normal((rows, 192), 6), normal((rows, 96), 7, 0.1)
    for call in (lambda s: mx.gated_quantize(z, axis=mx.MX_ROWWISE, status=s)[:1],
                 lambda s: mx.gated_backward_quantize(dh, z, axis=mx.MX_ROWWISE, status=s)[:1]):
        (got,), (right,) = ran_out(call, STAGES)
        check_lost(got, right, all_lost(got))


@pytest.mark.parametrize("counts,F", [([100, 0, 156], 96), ([5, 127, 128, 0, 0, 1000, 33, 2], 224)])
def test_gate_groups(counts, F):
    """Blocks of 32 rows of a segment that no row is in stay what they are, zeros."""
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    M = int(offs[-1])
    z, dh = normal((M, 2 * F), 8), normal((M, F), 9, 0.1)
    kw = dict(group_offsets=torch.from_numpy(offs).cuda(), col_capacity=mx.mx_grouped_padded_rows(offs))
    there = np.concatenate([np.arange(-(-n // 128) * 4) * 32 < n for n in counts])
    for call in (lambda s: mx.gated_quantize(z, status=s, **kw), lambda s: mx.gated_backward_quantize(dh, z, status=s, **kw)):
        (row, col), (row_right, col_right) = ran_out(call, STAGES)
        check_lost(row, row_right, all_lost(row))
        check_lost(col, col_right, np.broadcast_to(there, (col.rows, len(there))))


# every width of the token tile, contractions of one K block and of many, cut and whole
@pytest.mark.parametrize("with_status", [True, False])
@pytest.mark.parametrize("M,F,K", [(1, 40, 32), (1, 1408, 2048), (16, 333, 7168), (17, 1376, 992), (33, 520, 2048), (64, 1408, 1952),
                                   (128, 640, 7168), (333, 1408, 2048)])
def test_product_of_few_tokens(M, F, K, with_status):
    a, gate, up = (mx.quantize(normal((r, K), s, 0.1), mx.MX_ROWWISE)[0] for r, s in ((M, 1), (F, 2), (F, 3)))
    got, _ = ran_out(lambda s: mx.gemm_gated(a, gate, up, keep_preact=True, status=s), STAGES, with_status)
    assert all(torch.isnan(t).all() for t in got)


def test_taken_back_and_asked_once():
    """What was asked and taken back does not happen, and what was asked happens once (ran_out's last call)."""
    z = normal((64, 128), 6)
    want = mx.gated_quantize(z)[0]
    mx.mx_selftest_block_timeout(STAGES, LIMIT)
    mx.mx_selftest_block_timeout(0, 0)
    st = mx.new_status()
    row, _ = mx.gated_quantize(z, status=st)
    assert mx.read_status(st) == 0 and torch.equal(row.data, want.data)
    mx.mx_selftest_block_timeout(SUMS, LIMIT)                # the gate has no sums of rows: it runs as ever
    row, _ = mx.gated_quantize(z, status=st)
    assert mx.read_status(st) == 0 and torch.equal(row.data, want.data)
