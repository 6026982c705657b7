"""Host-side checks (no GPU): a state updated in place overlaps nothing else of its call."""
import pytest

import test_lm_abi as abi
from test_lm_abi import INVALID, addr, lib  # noqa: F401


@pytest.mark.parametrize("other", [dict(x=addr(6, 64)), dict(r=addr(6)), dict(i=addr(6, 4)), dict(decay=addr(6, 8)),
                                   dict(reset=addr(6, 17)), dict(y=addr(6)), dict(ckpt=addr(6))],
                         ids=["x", "r", "i", "decay", "reset", "y", "ckpt"])
def test_glr_state_in_place(lib, other):  # noqa: F811
    assert abi.glr_fwd(lib, h0=addr(6), h_last=addr(6), **other) == INVALID
    assert abi.glr_fwd(lib, h0=None, h_last=addr(6), **other) == INVALID
