"""INT8 mode serves from its quantised weights alone: moe_forward takes no bf16 w1 and w2 there, and in
every other mode refuses a call without them before it looks for a GPU."""
import ctypes

import pytest

from tests._util import ensure_built

m = ensure_built()
P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)


def _forward(precision, w1, w2):
    c = m.make_cfg(64, 512, 8, 2, 256, precision)
    s = m.moe_query(c)
    return m.lib().moe_forward(ctypes.byref(c), P, s.ring_slot, 0, P, P, P, w1, w2, P, s.wq or 1, P, P,
                               s.saved, P, s.workspace, None)


@pytest.mark.parametrize("precision", [m.MOE_PREC_BF16, m.MOE_PREC_MXFP8, m.MOE_PREC_MXFP4,
                                       m.MOE_PREC_FP8])
def test_other_modes_take_both(precision):
    for w1, w2 in ((None, P), (P, None), (None, None), (ODD, P), (P, ODD)):
        assert _forward(precision, w1, w2) == m.MOE_ERR_INVALID_ARG


def test_int8_mode_needs_neither():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up: without a GPU the call ends at the device check")
    for w1, w2 in ((None, None), (None, P), (P, None), (P, P)):
        assert _forward(m.MOE_PREC_INT8, w1, w2) not in (0, m.MOE_ERR_INVALID_ARG)
    for w1, w2 in ((ODD, None), (P, ODD)):
        assert _forward(m.MOE_PREC_INT8, w1, w2) == m.MOE_ERR_INVALID_ARG
