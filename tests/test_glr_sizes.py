"""Sizes of the recurrence's workspace for calls that are refused: none, whatever the numbers."""
import pytest

import kimi_delta_attention_23_b200 as kda
from kimi_delta_attention_23_b200 import build as kbuild


@pytest.mark.parametrize("T,batch,H,d", [(100, 2**31 - 1, 1, 8), (100, 2**30, 1, 8), (2**31 - 1025, 2**27, 1, 128),
                                         (100, 1, 2**31 - 1, 8), (2**31 - 1, 1, 1, 8), (-1, 1, 1, 8)])
def test_no_workspace_for_what_is_refused(T, batch, H, d):
    kbuild.build()
    assert kda.kda_glr_bwd_workspace_size(T, batch, H, d) == 0


@pytest.mark.parametrize("T,batch,H,d", [(100, 2**27 - 1, 1, 1), (2**31 - 1025, 1, 64, 128)])
def test_the_largest_ones_have_a_size(T, batch, H, d):
    kbuild.build()
    least = batch * H * (d + 1) * 4
    assert least <= kda.kda_glr_bwd_workspace_size(T, batch, H, d) <= 8 * least
