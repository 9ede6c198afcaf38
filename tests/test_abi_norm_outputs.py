"""The block norm's C entry point refuses an 8-bit h over rows that it still reads or writes: codes are a half or a
quarter as long as the rows, so they lie over other rows (no GPU needed)."""
import ctypes

import pytest

from test_abi_int8_norm import EINVAL, NORM, P, P2, call

P3, P4 = ctypes.c_void_p(0x300000), ctypes.c_void_p(0x400000)
APART = dict(NORM, x=P, y=P2, r=P3, h=P4)


@pytest.mark.parametrize("out", [1, 2, 3])
@pytest.mark.parametrize("changes", [dict(h=P), dict(h=P2), dict(h=P3), dict(y=None, post=None, gate=None, gate_kind=0, r=None, h=P)],
                         ids=["x", "y", "r", "x alone"])
def test_codes_over_rows_are_refused(out, changes):
    assert call("fg_block_norm", APART, out=out, **changes) == EINVAL
