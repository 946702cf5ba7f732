"""Refusals of the 4-bit cache and attention calls, on the host before any HIP
call (no GPU needed), and the binding's own checks."""
from __future__ import annotations

import ctypes as C

import pytest
import torch

import block_scoring_top_amd as bst

OK, ERR_NULL, ERR_ARG, ERR_WS = 0, -1, -2, -3
FAKE, ODD, NULL = C.c_void_p(0x1000), C.c_void_p(0x1008), None  # never dereferenced
WS = bst.ATTN_WORKSPACE_BYTES


def _store(**kw):
    a = dict(k=FAKE, v=FAKE, dtype=0, ld_k=256, ld_v=256, slots=FAKE, n=4, hkv=2, d=128, codes=FAKE, scales=FAKE,
             pages=1, stream=NULL)
    a.update(kw)
    return bst.lib().kv4_store(*a.values())


def _load(**kw):
    a = dict(codes=FAKE, scales=FAKE, pages=1, slots=FAKE, n=4, hkv=2, d=128, k=FAKE, v=FAKE, dtype=0, ld_k=256,
             ld_v=256, stream=NULL)
    a.update(kw)
    return bst.lib().kv4_load(*a.values())


@pytest.mark.parametrize("call", [_store, _load])
def test_kv4_refusals(call):
    assert call(n=0) == OK
    for kw in (dict(n=-1), dict(dtype=3), dict(dtype=-1), dict(d=96), dict(d=32, ld_k=64, ld_v=64), dict(hkv=0),
               dict(ld_k=255), dict(ld_v=248), dict(ld_k=260), dict(ld_v=258), dict(pages=0), dict(pages=-1),
               dict(hkv=1 << 14, ld_k=1 << 22, ld_v=1 << 22), dict(pages=1 << 25), dict(k=ODD), dict(v=ODD), dict(codes=ODD),
               dict(scales=ODD)):
        assert call(**kw) == ERR_ARG, kw
    for name in ("k", "v", "slots", "codes", "scales"):
        assert call(**{name: NULL}) == ERR_NULL, name


def _slots(**kw):
    a = dict(q=FAKE, dtype=0, ld_q=1024, rows=2, hq=8, hkv=2, d=128, c0=FAKE, c1=FAKE, form=1, ld_c=0, pages=4,
             slots=FAKE, ld_slots=2051, count=NULL, scale=0.1, out=FAKE, ld_out=1024, lse=NULL, ws=NULL, ws_bytes=0,
             stream=NULL)
    a.update(kw)
    return bst.lib().attn_slots(*a.values())


def _window(**kw):
    a = dict(q=FAKE, dtype=0, ld_q=1024, rows=2, hq=8, hkv=2, d=128, c0=FAKE, c1=FAKE, form=1, ld_c=0, pages=4, pt=FAKE,
             pt_stride=4, ptr=FAKE, req=1, pos=FAKE, max_rows=2, window=64, sinks=4, scale=0.1, out=FAKE, ld_out=1024,
             lse=NULL, ws=NULL, ws_bytes=0, stream=NULL)
    a.update(kw)
    return bst.lib().attn_window(*a.values())


@pytest.mark.parametrize("call", [_slots, _window])
def test_attention_refusals(call):
    assert call(rows=0) == OK
    for kw in (dict(rows=-1), dict(dtype=2), dict(dtype=-1), dict(form=2), dict(form=-1), dict(d=80), dict(hq=0),
               dict(hkv=0), dict(hq=7), dict(ld_q=1023), dict(ld_q=1028), dict(ld_out=1016), dict(ld_out=1025),
               dict(pages=0), dict(pages=-1), dict(pages=1 << 25), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=ODD),
               dict(out=ODD), dict(c0=ODD), dict(c1=ODD), dict(ws=ODD, ws_bytes=WS),
               dict(hq=1 << 14, ld_q=1 << 21, ld_out=1 << 21), dict(form=0, ld_c=255), dict(form=0, ld_c=260), dict(form=0, ld_c=(1 << 24) + 8)):
        assert call(**kw) == ERR_ARG, kw
    for name in ("q", "c0", "c1", "out"):
        assert call(**{name: NULL}) == ERR_NULL, name
    assert call(ws=FAKE, ws_bytes=WS - 1) == ERR_WS
    assert call(ws=FAKE, ws_bytes=0) == ERR_WS


def test_slots_refusals():
    assert _slots(ld_slots=-1) == ERR_ARG
    assert _slots(slots=NULL) == ERR_NULL
    assert _slots(rows=(1 << 20) + 1) == ERR_ARG  # more than 2^21 rows times kv heads


def test_window_refusals():
    assert _window(req=0) == OK
    assert _window(max_rows=0) == OK
    for kw in (dict(req=-1), dict(max_rows=-1), dict(window=-1), dict(sinks=-1), dict(pt_stride=0),
               dict(req=1 << 23, max_rows=8)):
        assert _window(**kw) == ERR_ARG, kw
    for name in ("pt", "ptr", "pos"):
        assert _window(**{name: NULL}) == ERR_NULL, name


def test_workspace_size_matches_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "blockscore.h")).read()
    m = re.search(r"BS_ATTN_WORKSPACE_BYTES \(\(\(size_t\)(\d+) << (\d+)\) \+ \(\(size_t\)(\d+) << (\d+)\)\)", text)
    a, b, c, d = map(int, m.groups())
    assert (a << b) + (c << d) == WS


def test_binding_checks_cpu_tensors_and_shapes():
    cache = bst.KV4Cache.empty(1, 2, 64, "cpu")
    assert (cache.kv_heads, cache.head_dim, cache.num_pages) == (2, 64, 1)
    k = torch.zeros(3, 2, 64)
    s = torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # CPU tensors
        bst.kv4_store(k, k, s, cache)
    with pytest.raises(ValueError):
        bst.kv4_load(cache, s, k, k)
    with pytest.raises(ValueError):
        bst.attn_slots(q, cache, s.view(3, 1), torch.zeros_like(q))
    with pytest.raises(ValueError):
        bst.kv4_store(k[:, :1], k[:, :1], s, cache)  # heads
    with pytest.raises(ValueError):
        bst.kv4_store(k, k, s[:2], cache)
    with pytest.raises(ValueError):
        bst.attn_slots(q[:, :3], cache, s.view(3, 1), q[:, :3])  # 3 heads over 2
    with pytest.raises(ValueError):
        bst.attn_slots(q, cache, s.view(3, 1), q[:2])
    with pytest.raises(ValueError):
        bst.KV4Cache(torch.zeros(65, 2, 2, 32, dtype=torch.uint8), torch.zeros(65, 2, 2, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        bst.KV4Cache(torch.zeros(64, 2, 2, 32, dtype=torch.uint8), torch.zeros(64, 2, 2, 4, dtype=torch.uint8))
    with pytest.raises(ValueError):
        bst.KV16Cache(torch.zeros(64, 2, 64), torch.zeros(64, 2, 128))


def test_bounds_past_32_bits_are_the_largest():
    """A bound on positions or rows is not wrapped to 32 bits; negative ones stay refused."""
    got = [bst._int32(x) for x in (0, 5, 2**31 - 1, 2**31, 1 << 32, 1 << 40, -1, -(1 << 32))]
    assert got == [0, 5, 2**31 - 1, 2**31 - 1, 2**31 - 1, 2**31 - 1, -1, -1]


def test_the_reference_rounds_to_the_nearest_code():
    """The tests' own quantiser, at the halfway points and the ends."""
    import numpy as np
    from attn_ref import dequantise, quantise
    x = np.zeros(32)
    x[:16] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -0.75, 0.2500001, 0.7499999, -5.0000001, 6.5, 0.0]
    x[16] = 7.5
    c, s = quantise(x)
    assert s[0] == 127
    want = [4, 0, 1, 1, 2, 2, 4, 4, 6, 0, -1, 0.5, 0.5, -6, 6, 0, 6]
    assert np.array_equal(dequantise(c, s)[:17], want)
    for v, byte in ((0.0, 7), (2.0 ** -130, 7), (2.0 ** 127, 252), (np.inf, 255), (np.nan, 255), (8.0, 128), (7.99, 127)):
        assert quantise(np.full(32, v))[1][0] == byte, v
