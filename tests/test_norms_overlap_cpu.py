"""The gated norm's backward on the CPU: gradients that share addresses in one buffer are refused (nothing here is launched)."""
import pytest

from selective_state_space_62_amd import binding as b
from test_blocks_cpu import INVALID, at, gated

ROWS = (2560, 256, 40)                                     # three heads of 40 in rows of 256


@pytest.mark.parametrize("apart,dzs", [
    (0, ROWS), (39, ROWS), (40, ROWS), (80, ROWS), (119, ROWS), (137, ROWS), (255, ROWS),   # heads, or the next row, reached
    (120, (2560, 128, 40)), (120, (1280, 256, 40)), (120, (2560, 256, 49)),                    # other strides (of 48 the last head ends with the row)
    (2560, ROWS),                                                                              # the next batch row
])
def test_columns_that_meet(apart, dzs):
    st, msg = gated("bwd", dxs=ROWS, dz=at(5, 2 * apart), dzs=dzs)
    assert st == INVALID and "dz" in msg, (st, msg)


def test_half_an_element_apart():
    st, msg = gated("bwd", io=b.SS_F32, dxs=ROWS, dz=at(5, 4 * 120 + 2), dzs=ROWS)
    assert st == INVALID and "dz" in msg, (st, msg)
