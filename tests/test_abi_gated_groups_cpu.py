"""Host-side checks of the gate's groups (no GPU needed): what the kernel alone would
find, and could report through a status word only, is refused where the host can see it."""
import pytest

import mxfp8_block_scaled_gb300 as mx
from tests.test_abi_gated_cpu import INVALID, SHAPE, L, gate, status_of  # noqa: F401 (a fixture)

GROUPS = dict(group_offsets=0x9000, n_groups=4)


def quantizer(**kw):
    d = dict(x=0x1000, rows=32, cols=64, ldx=64, axis=mx.MX_BOTH, row_data=0x10000, row_scale=0x20000, col_data=0x30000,
             col_scale=0x40000, group_offsets=0x9000, n_groups=4, col_capacity=512, dev_status=None, stream=None)
    d.update(kw)
    return status_of(mx.mx_quantize, *d.values())


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("axis", [mx.MX_COLWISE, mx.MX_BOTH])
def test_capacity_of_nothing(back, axis):
    """Rows, and no room for them: refused as by the quantiser; without rows there is nothing to refuse."""
    assert gate(back, **GROUPS, axis=axis, col_capacity=0) == SHAPE == quantizer(axis=axis, col_capacity=0)
    assert gate(back, **GROUPS, axis=axis, col_capacity=0, rows=0) == 0 == quantizer(axis=axis, col_capacity=0, rows=0)
    assert gate(back, **GROUPS, axis=axis, col_capacity=0, f=0) == 0


@pytest.mark.parametrize("back", [False, True])
def test_capacity_of_no_whole_segments(back):
    for bad in (-128, 100, 127):
        assert gate(back, **GROUPS, col_capacity=bad) == INVALID
