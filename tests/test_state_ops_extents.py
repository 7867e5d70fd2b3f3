"""Extents that 32 bits do not hold.  The C ABI counts slots, heads, channels and entries in int32, and ctypes
passes a larger number without its upper bits: a pool of 2^32 + 8 slots would be taken for one of 8."""
import pytest
import torch

import kimi_delta_attention_23_b200 as kda
from kimi_delta_attention_23_b200 import pool

BIG = 2**32 + 8


class Stand:
    """A CUDA tensor as far as the checks look at one."""

    def __init__(self, *shape, dtype=torch.float32):
        self.shape, self.dtype, self.is_cuda = shape, dtype, True

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n


def test_extents_beyond_32_bits_are_refused():
    for shape in ((1, 1, BIG), (1, BIG, 1), (BIG, 1, 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            kda._where(Stand(*shape), "x", 3)
        with pytest.raises(ValueError, match="2\\^31"):
            kda._need_rank(Stand(*shape), "state_pool", torch.float32, 3, None, 0)
    assert kda._where(Stand(1, 2, 2**31 - 1), "x", 3)[1] == (1, 2, 2**31 - 1)
    for shape, stacked in (((BIG, 3), False), ((2, BIG, 3), True), ((BIG, 2, 3), True)):
        with pytest.raises(ValueError, match="2\\^31"):
            pool._layout(Stand(*shape), stacked)
    # what lies behind the slot's index is counted in 64 bits
    assert pool._layout(Stand(2, BIG), False)[2:] == (1, 2, BIG)


@pytest.mark.gpu
def test_a_pool_of_more_slots_than_32_bits_count():
    many = torch.empty(BIG, 1, 1, device="cuda")  # 17 GB, never touched
    ints = torch.zeros(1, dtype=torch.int32, device="cuda")
    one, cell = torch.zeros(1, 1, device="cuda"), torch.zeros(1, 1, 1, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        kda.kda_pool_copy(many, ints, ints)
    with pytest.raises(ValueError, match="2\\^31"):
        kda.kda_glr_decode(cell, cell, one, one[0], one, many, ints)
    with pytest.raises(ValueError, match="2\\^31"):
        kda.kda_tree_decode(cell, cell, cell, cell, one, one[0], one, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                            ints - 1, many[:, None], ints)
