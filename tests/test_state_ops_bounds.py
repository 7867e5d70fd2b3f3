"""The safe gate's lower bound: a gate is the logarithm of a decay, so a bound above 0 (or one that is not a number)
is refused by the calls whose exponential is made for gates of at most 0."""
import ctypes

import pytest

import kimi_delta_attention_23_b200 as kda
from kimi_delta_attention_23_b200 import build as kbuild

OK, INVALID = 0, 1
SAFE = kda.GATE_SAFE


@pytest.mark.parametrize("flags,bound,code", [(SAFE, 0.5, INVALID), (SAFE, float("inf"), INVALID), (SAFE, float("nan"), INVALID),
                                              (SAFE, 0.0, OK), (SAFE, float("-inf"), OK), (0, 0.5, OK), (0, float("nan"), OK)])
def test_bounds(flags, bound, code):
    kbuild.build()
    lib, p = kda.load_library(), ctypes.c_void_p(256)
    # empty batches: nothing is launched
    assert lib.kda_glr_fwd(p, 1, p, 1, p, p, p, p, 0, 0, 2, 128, p, 4, p, p, 1, None, flags, bound, None, None) == code
    assert lib.kda_glr_decode(p, 1, p, 1, p, p, p, 0, 2, 128, p, 4, p, p, 1, flags, bound, None, None) == code
    assert lib.kda_tree_decode(p, p, p, 1, p, p, p, p, p, p, 0, 0, 8, 2, 2, 128, 128, p, 4, p, p, 1, p, flags, bound, None, None) == code
    assert lib.kda_tree_commit(p, 1, p, p, p, p, p, p, p, 0, 0, 8, 2, 2, 128, 128, p, 4, p, flags, bound, None, None) == code
    if code != OK:  # (an empty batch of gradients is written on the device)
        assert lib.kda_glr_bwd(p, 1, p, 1, p, 1, p, p, p, p, 0, 0, 2, 128, p, p, p, p, p, p, p, p, flags, bound, p, 0, None, None) == code
