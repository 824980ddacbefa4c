"""Rope's own choices, without a GPU (the table stays on the host)."""
import math

import pytest

from decoder_greedy_decode_b200.rotary import Rope


def rope(scaling, factor, **kw):
    return Rope(64, scaling=scaling, factor=factor, orig_ctx=8192.0, device="cpu", **kw)


@pytest.mark.parametrize("factor", [0.25, 0.5, 1.0])
def test_by_parts_magnitude_is_1_up_to_a_factor_of_1(factor):
    assert rope("parts", factor).mscale == 1.0
    assert rope("parts", factor).c.mscale == 1.0


def test_by_parts_magnitude_above_1():
    for factor in (1.5, 4.0, 32.0):
        assert rope("parts", factor).mscale == 0.1 * math.log(factor) + 1.0
    assert rope("parts", 4.0, mscale=0.75).mscale == 0.75
    assert rope("linear", 4.0).mscale == 1.0 and rope("ntk", 0.5).mscale == 1.0
