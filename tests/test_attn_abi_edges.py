"""Refusals of the attention calls at the ends of their arguments' ranges, on the
host before any HIP call (no GPU needed)."""
from __future__ import annotations

import pytest

from test_attn_abi import ERR_ARG, OK, _slots, _window


@pytest.mark.parametrize("call", [_slots, _window])
def test_scales_beyond_2_to_the_127_are_refused(call):
    """Times log2(e) they would be infinite, and a score of 0 a NaN."""
    for scale in (3.4028234e38, -3.4028234e38, 1.8e38, float("inf"), -float("inf"), float("nan")):
        assert call(scale=scale) == ERR_ARG, scale
    for scale in (2.0 ** 127, -(2.0 ** 127), 0.0, 1e-45):
        assert call(scale=scale, rows=0) == OK, scale
