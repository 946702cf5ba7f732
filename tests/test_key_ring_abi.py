"""Refusals of the key compression with a ring of any depth (no GPU needed)."""
from __future__ import annotations

import ctypes as C

import pytest
import torch

import block_scoring_top_amd as bst
from block_scoring_top_amd.pipeline import PagedBatch

OK, ERR_NULL, ERR_ARG = 0, -1, -2
FAKE, NULL = C.c_void_p(0x1000), None  # never dereferenced


def _call(fn, **kw):
    a = dict(k=FAKE, n=4, ptr=FAKE, start=FAKE, mrope=NULL, req=1, most=4, rot=128, t=16, h=24, w=24, theta=1e6, ring=FAKE,
             ring_pos=NULL, slots=16, pt=FAKE, pt_stride=2, codes=FAKE)
    a.update(dict(scales=FAKE) if fn.startswith("idx4") else {}, pages=4, stream=NULL)
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(bst.lib(), fn)(*a.values())


@pytest.mark.parametrize("fn", ["idx_compress_store_ring", "idx4_compress_store_ring"])
def test_refusals(fn):
    assert _call(fn, n=0, most=0) == OK and _call(fn, req=0) == OK
    for slots in (0, -4, 1, 2, 3, 5, 12, 24, 1 << 17, -2**31):
        assert _call(fn, slots=slots) == ERR_ARG, slots
        assert _call(fn, slots=slots, req=0) == ERR_ARG, slots
    for kw in (dict(n=-1), dict(req=-1), dict(req=65536), dict(most=5), dict(rot=127), dict(t=17), dict(theta=0.0),
               dict(pt_stride=0), dict(pages=0)):
        assert _call(fn, **kw) == ERR_ARG, kw
    for name in ("k", "ptr", "start", "ring", "pt", "codes"):
        assert _call(fn, **{name: NULL}) == ERR_NULL, name
    assert _call(fn, mrope=FAKE) == ERR_NULL


@pytest.mark.parametrize("most_cut,slots", [(0, 4), (1, 4), (2, 8), (5, 8), (6, 16), (13, 16), (14, 32)])
def test_key_ring_of_a_batch(most_cut, slots):
    batch = PagedBatch(3, 200, 9, 12, "cpu")
    ring, pos = batch.key_ring(most_cut)
    assert ring.shape == (3, slots, 128) and ring.dtype == torch.bfloat16 and pos is None
    assert batch.key_ring(most_cut, mrope=True)[1].shape == (3, slots // 4, 3)


def test_binding_checks():
    z = dict(dtype=torch.int32)
    k, ptr, start, table = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(2, **z), torch.zeros(1, **z), torch.zeros(1, 2, **z)
    cache = torch.zeros(32, 128, dtype=torch.bfloat16)
    for ring, pos in ((torch.zeros(1, 2, 128), None), (torch.zeros(2, 8, 128), None), (torch.zeros(1, 8, 64), None),
                      (torch.zeros(4, 128), None), (torch.zeros(1, 8, 128), torch.zeros(1, 3, **z)),
                      (torch.zeros(1, 8, 128), torch.zeros(1, 1, 3, **z)), (torch.zeros(1, 4, 128), torch.zeros(1, 2, 3, **z))):
        with pytest.raises(ValueError):
            bst.idx_compress_store(k, ptr, start, None, 4, 128, (16, 24, 24), 1e6, ring.bfloat16(), pos, table, cache, 2)
        with pytest.raises(ValueError):
            bst.idx4_compress_store(k, ptr, start, None, 4, 128, (16, 24, 24), 1e6, ring.bfloat16(), pos, table,
                                    bst.Idx4Cache.empty(2, 4, "cpu"))
