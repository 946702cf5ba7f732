"""Refusals of the page table, 8-bit cache and 4-bit index calls, on the host
before any HIP call (no GPU needed), the binding's own checks, and the tests' own
references at known points."""
from __future__ import annotations

import ctypes as C

import numpy as np
import pytest
import torch

import block_scoring_top_amd as bst
from more_ref import E4M3, Kv8, e4m3_round, e4m3_value, kv8_exponent, pages_extend, pages_release

OK, ERR_NULL, ERR_ARG, ERR_WS = 0, -1, -2, -3
FAKE, ODD, NULL = C.c_void_p(0x1000), C.c_void_p(0x1008), None  # never dereferenced


def _call(fn, defaults):
    def call(**kw):
        a = dict(defaults)
        assert set(kw) <= set(a)
        a.update(kw)
        return getattr(bst.lib(), fn)(*a.values())
    return call


_store8 = _call("kv8_store", dict(k=FAKE, v=FAKE, dtype=0, ld_k=256, ld_v=256, slots=FAKE, n=4, hkv=2, d=128, codes=FAKE,
                                  scales=FAKE, pages=1, stream=NULL))
_load8 = _call("kv8_load", dict(codes=FAKE, scales=FAKE, pages=1, slots=FAKE, n=4, hkv=2, d=128, k=FAKE, v=FAKE, dtype=0,
                                ld_k=256, ld_v=256, stream=NULL))


@pytest.mark.parametrize("call", [_store8, _load8])
def test_kv8_refusals(call):
    assert call(n=0) == OK
    for kw in (dict(n=-1), dict(dtype=3), dict(dtype=-1), dict(d=96), dict(d=32, ld_k=64, ld_v=64), dict(hkv=0),
               dict(ld_k=255), dict(ld_v=248), dict(ld_k=260), dict(ld_v=258), dict(pages=0), dict(pages=-1),
               dict(hkv=1 << 14, ld_k=1 << 22, ld_v=1 << 22), dict(pages=1 << 25), dict(k=ODD), dict(v=ODD),
               dict(codes=ODD), dict(scales=ODD)):
        assert call(**kw) == ERR_ARG, kw
    for name in ("k", "v", "slots", "codes", "scales"):
        assert call(**{name: NULL}) == ERR_NULL, name


_slots8 = _call("attn_slots", dict(q=FAKE, dtype=0, ld_q=1024, rows=2, hq=8, hkv=2, d=128, c0=FAKE, c1=FAKE, form=8, ld_c=0,
                                   pages=4, slots=FAKE, ld_slots=2051, count=NULL, scale=0.1, out=FAKE, ld_out=1024,
                                   lse=NULL, ws=NULL, ws_bytes=0, stream=NULL))
_window8 = _call("attn_window", dict(q=FAKE, dtype=0, ld_q=1024, rows=2, hq=8, hkv=2, d=128, c0=FAKE, c1=FAKE, form=8,
                                     ld_c=0, pages=4, pt=FAKE, pt_stride=4, ptr=FAKE, req=1, pos=FAKE, max_rows=2,
                                     window=64, sinks=4, scale=0.1, out=FAKE, ld_out=1024, lse=NULL, ws=NULL, ws_bytes=0,
                                     stream=NULL))


@pytest.mark.parametrize("call", [_slots8, _window8])
def test_attention_over_8_bits_refusals(call):
    assert call(rows=0) == OK
    for kw in (dict(rows=-1), dict(dtype=2), dict(form=7), dict(form=16), dict(d=80), dict(hq=7), dict(ld_q=1028),
               dict(pages=0), dict(pages=1 << 25), dict(scale=float("nan")), dict(c0=ODD), dict(c1=ODD)):
        assert call(**kw) == ERR_ARG, kw
    for name in ("q", "c0", "c1", "out"):
        assert call(**{name: NULL}) == ERR_NULL, name


_store4 = _call("idx4_store", dict(keys=FAKE, dtype=0, ld=128, slots=FAKE, n=4, codes=FAKE, scales=FAKE, keys_in=64,
                                   stream=NULL))
_load4 = _call("idx4_load", dict(codes=FAKE, scales=FAKE, keys_in=64, slots=FAKE, n=4, keys=FAKE, dtype=0, ld=128,
                                 stream=NULL))


@pytest.mark.parametrize("call", [_store4, _load4])
def test_idx4_refusals(call):
    assert call(n=0) == OK
    for kw in (dict(n=-1), dict(dtype=3), dict(dtype=-1), dict(ld=127), dict(ld=132), dict(ld=120), dict(keys_in=0),
               dict(keys_in=-1), dict(keys_in=1 << 31), dict(keys=ODD), dict(codes=ODD), dict(scales=ODD)):
        assert call(**kw) == ERR_ARG, kw
    for name in ("keys", "slots", "codes", "scales"):
        assert call(**{name: NULL}) == ERR_NULL, name


_score4 = _call("idx4_score", dict(q=FAKE, codes=FAKE, scales=FAKE, pages=4, pt=FAKE, pt_stride=4, ptr=FAKE, req=1,
                                   pos=FAKE, rows=2, c=4, max_vis=64, scores=FAKE, ld=64, row_len=NULL, stream=NULL))


def test_idx4_score_refusals():
    assert _score4(rows=0) == OK and _score4(req=0) == OK
    for kw in (dict(rows=-1), dict(req=-1), dict(c=2), dict(c=0), dict(max_vis=-1), dict(pages=0), dict(pages=1 << 25),
               dict(pt_stride=0), dict(ld=63), dict(max_vis=65, ld=65), dict(req=65536), dict(q=ODD), dict(codes=ODD),
               dict(scales=ODD), dict(max_vis=65535 * 4096 + 1, ld=1 << 29, pt_stride=1 << 25)):
        assert _score4(**kw) == ERR_ARG, kw
    for name in ("q", "codes", "scales", "pt", "ptr", "pos", "scores"):
        assert _score4(**{name: NULL}) == ERR_NULL, name


_compress4 = _call("idx4_compress_store", dict(k=FAKE, n=4, ptr=FAKE, start=FAKE, mrope=NULL, req=1, most=4, rot=128, t=16,
                                               h=24, w=24, theta=1e6, ring=FAKE, ring_pos=NULL, pt=FAKE, pt_stride=2,
                                               codes=FAKE, scales=FAKE, pages=4, stream=NULL))


def test_idx4_compress_refusals():
    assert _compress4(n=0, most=0) == OK and _compress4(req=0) == OK and _compress4(most=0) == OK
    for kw in (dict(n=-1), dict(req=-1), dict(req=65536), dict(most=5), dict(rot=127), dict(t=17), dict(theta=0.0),
               dict(theta=float("nan")), dict(pt_stride=0), dict(pages=0), dict(pages=-1), dict(codes=ODD),
               dict(scales=ODD)):
        assert _compress4(**kw) == ERR_ARG, kw
    for name in ("k", "ptr", "start", "ring", "pt", "codes", "scales"):
        assert _compress4(**{name: NULL}) == ERR_NULL, name
    assert _compress4(mrope=FAKE) == ERR_NULL


_PAGES = dict(kv_len=FAKE, held=FAKE, change=FAKE, req=2, pt=FAKE, pt_stride=4, ring=FAKE, size=8, pool=FAKE, kv_out=FAKE,
              held_out=FAKE, pool_out=FAKE)
_extend = _call("pages_extend", dict(**_PAGES, ptr=FAKE, start=NULL, pos=FAKE, slots=FAKE, rows=4, stream=NULL))
_release = _call("pages_release", dict(**_PAGES, stream=NULL))


@pytest.mark.parametrize("call", [_extend, _release])
def test_pages_refusals(call):
    for kw in (dict(req=-1), dict(pt_stride=0), dict(size=0), dict(size=1 << 25)):
        assert call(**kw) == ERR_ARG, kw
    for name in _PAGES:
        if name not in ("req", "pt_stride", "size"):
            assert call(**{name: NULL}) == ERR_NULL, name
    if call is _extend:
        assert call(rows=-1) == ERR_ARG
        for name in ("ptr", "pos", "slots"):
            assert call(**{name: NULL}) == ERR_NULL, name


def test_binding_checks():
    cache = bst.KV8Cache.empty(1, 2, 64, "cpu")
    assert (cache.kv_heads, cache.head_dim, cache.num_pages) == (2, 64, 1)
    assert cache.scales[0, 0, 0].item() == 2.0 ** -120
    k, s = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        bst.kv8_store(k, k, s, bst.KV4Cache.empty(1, 2, 64, "cpu"))
    with pytest.raises(TypeError):
        bst.kv4_store(k, k, s, cache)
    for bad in (lambda: bst.kv8_store(k, k, s, cache), lambda: bst.kv8_load(cache, s, k, k),          # CPU tensors
                lambda: bst.kv8_store(k[:, :1], k[:, :1], s, cache), lambda: bst.kv8_store(k, k, s[:2], cache),
                lambda: bst.KV8Cache(torch.zeros(65, 2, 2, 64, dtype=torch.uint8), torch.zeros(1, 2, 2)),
                lambda: bst.KV8Cache(torch.zeros(64, 2, 2, 64, dtype=torch.uint8), torch.zeros(2, 2, 2))):
        with pytest.raises(ValueError):
            bad()
    keys = bst.Idx4Cache.empty(2, 4, "cpu")
    assert (keys.num_keys, keys.num_pages, keys.c) == (32, 2, 4)
    x = torch.zeros(3, 128)
    with pytest.raises(TypeError):
        bst.idx4_store(x, s, cache)
    for bad in (lambda: bst.idx4_store(x, s, keys), lambda: bst.idx4_load(keys, s, x), lambda: bst.idx4_store(x, s[:2], keys),
                lambda: bst.idx4_store(x[:, :64], s, keys), lambda: bst.Idx4Cache.empty(2, 2, "cpu"),
                lambda: bst.Idx4Cache(torch.zeros(17, 64, dtype=torch.uint8), torch.zeros(17, 4, dtype=torch.uint8), 4),
                lambda: bst.Idx4Cache(torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(16, 8, dtype=torch.uint8), 4)):
        with pytest.raises(ValueError):
            bad()
    pool = bst.PagePool.full(8, "cpu")
    assert pool.state.tolist() == [0, 8, 0, 0] and pool.ring.tolist() == list(range(8))
    n, t = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    for bad in (lambda: bst.pages_release(pool, n, n, n, t), lambda: bst.pages_release(pool, n, n, n[:1], t),
                lambda: bst.pages_release(pool, n, n, n, t[:1]),
                lambda: bst.pages_release(pool, n, n, n, t, pool_out=bst.PagePool.full(8, "cpu")),
                lambda: bst.PagePool(n, n)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        bst.pages_release(n, n, n, n, t)


def test_the_references_at_known_points():
    assert E4M3[126] == 448 and E4M3[1] == 2.0 ** -9 and E4M3[8] == 2.0 ** -6 and E4M3[56] == 1.0
    got = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(e4m3_value(np.arange(256)), got)
    for x, want in ((1.0625, 1.0), (1.1875, 1.25), (2.0 ** -10, 0.0), (3 * 2.0 ** -10, 2.0 ** -8), (-432.0, -448.0), (447, 448),
                    (424.0, 416.0), (0.0, 0.0)):
        assert e4m3_value(e4m3_round(np.array([x])))[0] == want, x
    for top, e in ((448.0, 0), (448.0001, 1), (256.0, 0), (224.0, -1), (225.0, 0), (0.0, -120), (2.0 ** -130, -120), (1e38, 118),
                   (3.39e38, 119)):
        assert kv8_exponent(top) == e, top
    c = Kv8(1, 1, 64)
    x = np.full((1, 1, 64), 448.0)
    c.store(x, x, np.array([3]))
    c.store(8 * x, x, np.array([4]))
    k, v = c.values()
    assert (k[3] == 448).all() and (k[4] == 3584).all() and c.exps.ravel().tolist() == [3, 0]
    c.store(x / 8, x, np.array([0]))                              # begun anew
    assert c.exps.ravel().tolist() == [-3, 0]
    r = pages_extend([0, 64, 3], [0, 1, 1], [65, 1, 0], np.array([[-1, -1], [7, -1], [9, -1]]), np.array([4, 5, 6, 8]),
                     [3, 4, 0, 0], 70)
    assert r["pool"] == [2, 1, 0, 0] and r["table"].tolist() == [[8, 4], [7, 5], [9, -1]] and r["ptr"] == [0, 65, 66, 66]
    assert r["slots"][:2] == [512, 513] and r["slots"][64:] == [256, 320, -1, -1, -1, -1] and r["pos"][64:66] == [64, 64]
    r = pages_release(r["kv_len"], r["held"], [64, 0, -1], r["table"], np.array([4, 5, 6, 8]), r["pool"])
    assert r["table"].tolist() == [[8, -1], [-1, -1], [9, -1]] and r["ring"].tolist() == [7, 5, 6, 4]
    assert r["pool"] == [2, 4, 0, 0] and r["held"] == [1, 0, 1]
