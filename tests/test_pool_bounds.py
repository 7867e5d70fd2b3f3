"""The largest lists and pools that a plan may walk: its 1024 threads count a step past the end in 32 bits."""
import ctypes

import pytest

import kimi_delta_attention_23_b200 as kda
from kimi_delta_attention_23_b200 import build as kbuild

INVALID, WORKSPACE = 1, 3
MOST = 2**31 - 1


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


@pytest.mark.parametrize("n,slots,code", [(MOST, 8, INVALID), (MOST - 1023, 8, INVALID), (4, MOST, INVALID),
                                          (4, MOST - 1023, INVALID), (MOST - 1024, 8, WORKSPACE), (4, MOST - 1024, WORKSPACE)])
def test_lists_and_pools_that_would_be_walked_past_2_31(lib, n, slots, code):
    p = ctypes.c_void_p(256)
    no_work = (None, 0, None, None)  # what is not refused for its size comes as far as the missing workspace
    assert lib.kda_pool_fork(p, 1, slots, 1, p, p, p, n, *no_work) == code
    assert lib.kda_pool_free(p, 1, slots, 1, p, p, n, *no_work) == code
    assert lib.kda_pool_compact(p, 1, slots, 1, p, p, n, p, *no_work) == code
