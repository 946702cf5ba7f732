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


@pytest.mark.parametrize("rows,req,max_rows", [(2**31 - 1, 2**31 - 1, 2**31 - 1), (2**31 - 1, 2**31 - 1, 2**27),
                                               (2**30, 2**31 - 1, 2**30), (2**26, 2**31 - 1, 2**26)])
@pytest.mark.parametrize("d,hq,hkv", [(64, 1 << 14, 1 << 14), (64, 1 << 14, 1 << 13), (256, 1 << 12, 1 << 12), (64, 1 << 14, 1)])
@pytest.mark.parametrize("form", [0, 1])
def test_the_largest_products_of_requests_rows_and_heads_are_refused(rows, req, max_rows, d, hq, hkv, form):
    """Tiles times heads past 2^63 do not wrap to a number of workgroups."""
    assert _window(rows=rows, req=req, max_rows=max_rows, d=d, hq=hq, hkv=hkv, ld_q=hq * d, ld_out=hq * d, form=form,
                   ld_c=hkv * d, pt_stride=1 << 20, window=2**31 - 1) == ERR_ARG
