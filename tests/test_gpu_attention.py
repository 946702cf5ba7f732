"""The 4-bit cache and the attention calls on the GPU against the 64-bit
references of attn_ref.py (bounds derived there): types, head layouts, key
counts around every step of the kernels, strides, padding, empty rows, masks
over infinities and NaN, pools past 4 GiB, streams, graphs, and a run of the
whole path."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scoring_top_amd as bst
from attn_ref import attend_row, check_rows, dequantise, quantise
from gpu_util import say

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


# ---------------------------------------------------------------- the cache

def _store_case(T, hkv, d, kind, pad, seed, fused):
    g = _gen(seed)
    pages = -(-T // 64) + 2
    x = torch.randn((T, 3 * hkv, d), generator=g, device="cuda") * torch.exp(2 * torch.randn((T, 3 * hkv, 1), generator=g, device="cuda"))
    x = x.to(TYPES[kind])
    k, v = (x[:, hkv:2 * hkv], x[:, 2 * hkv:]) if fused else (x[:, hkv:2 * hkv].contiguous(), x[:, 2 * hkv:].contiguous())
    slots = torch.randperm(pages * 64, generator=g, device="cuda", dtype=torch.int32)[:T].contiguous()
    if pad:
        slots[::pad] = -1
        slots[T // 2] = pages * 64  # past the pool: skipped
    return k, v, slots, pages


@pytest.mark.parametrize("T,hkv,d,kind,pad,fused", [
    (1, 1, 64, "bf16", 0, False), (1, 8, 256, "f32", 0, True), (3, 5, 64, "f16", 0, True), (64, 2, 128, "bf16", 0, True),
    (65, 3, 128, "f16", 7, False), (257, 1, 256, "bf16", 5, True), (1003, 5, 64, "f32", 11, True), (2050, 2, 128, "f32", 3, False),
    (513, 7, 128, "bf16", 0, False),
    (16411, 4, 128, "f16", 0, False)])  # enough for the kernel's several-pieces form, and a part of one
def test_store_and_load_match_the_definition(T, hkv, d, kind, pad, fused):
    say(f"kv4 T={T} hkv={hkv} d={d} {kind} pad={pad} fused={fused}")
    k, v, slots, pages = _store_case(T, hkv, d, kind, pad, T * 7 + hkv, fused)
    cache = bst.KV4Cache(torch.full((pages * 64, hkv, 2, d // 2), 0xA5, dtype=torch.uint8, device="cuda"),
                         torch.full((pages * 64, hkv, 2, d // 32), 0x5A, dtype=torch.uint8, device="cuda"))
    bst.kv4_store(k, v, slots, cache)
    torch.cuda.synchronize()
    codes, scales, at = cache.codes.cpu().numpy(), cache.scales.cpu().numpy(), slots.cpu().numpy()
    want_c, want_s = np.full_like(codes, 0xA5), np.full_like(scales, 0x5A)
    there = (at >= 0) & (at < pages * 64)
    for i, x in enumerate((k, v)):
        c, s = quantise(_f64(x))
        want_c[at[there], :, i], want_s[at[there], :, i] = c[there], s[there]
    np.testing.assert_array_equal(scales, want_s)
    np.testing.assert_array_equal(codes, want_c)
    # read back: the slots in another order, one of them twice, with padding
    order = torch.randperm(T, generator=_gen(3), device="cuda")
    rd = torch.cat([slots[order], slots[:1]]).contiguous()
    for out_kind in ("bf16", "f16", "f32"):
        out = torch.full((T + 1, 2 * hkv + 1, d), 7.0, dtype=TYPES[out_kind], device="cuda")
        ko, vo = out[:, :hkv], out[:, hkv:2 * hkv]
        bst.kv4_load(cache, rd, ko, vo)
        torch.cuda.synchronize()
        r = rd.cpu().numpy()
        ok = (r >= 0) & (r < pages * 64)
        for i, o in enumerate((ko, vo)):
            want = np.zeros((T + 1, hkv, d))
            want[ok] = dequantise(want_c[r[ok]][:, :, i], want_s[r[ok]][:, :, i])
            want = torch.from_numpy(want).to(TYPES[out_kind])  # one rounding, of values that are mostly exact
            np.testing.assert_array_equal(_f64(o), _f64(want))
        assert (out[:, 2 * hkv:] == 7.0).all()  # what lies between the rows is left alone


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_store_special_values(kind):
    """Halfway values, saturation, zeros of both signs, subnormals, the ends of
    the range, infinities and NaN, one group each."""
    t = TYPES[kind]
    f = torch.finfo(t)
    rows = []
    base = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.5, 7.5, -0.25, -0.75, -1.25, -5.0, 0.0, -0.0])
    for scale in (1.0, 2.0 ** -9, 2.0 ** 12):
        rows.append(torch.nn.functional.pad(base * scale, (0, 32 - base.numel())))
    rows.append(torch.zeros(32))
    rows.append(-torch.zeros(32))
    rows.append(torch.full((32,), f.smallest_normal / 4))
    rows.append(torch.full((32,), f.max))
    rows.append(torch.cat([torch.full((1,), f.max), torch.full((31,), 1.0)]))
    for bad in (float("inf"), -float("inf"), float("nan")):
        r = torch.linspace(-3, 3, 32)
        r[17] = bad
        rows.append(r)
    rows.append(torch.linspace(-1, 1, 32))
    x = torch.stack(rows).to(t)                                   # 12 groups -> 3 heads of 128
    x = x.reshape(1, 3, 128).cuda()
    cache = bst.KV4Cache.empty(1, 3, 128, "cuda")
    slots = torch.tensor([5], dtype=torch.int32, device="cuda")
    bst.kv4_store(x, -x, slots, cache)
    torch.cuda.synchronize()
    for i, y in enumerate((x, -x)):
        c, s = quantise(_f64(y))
        np.testing.assert_array_equal(cache.scales[5:6, :, i].cpu().numpy(), s)
        np.testing.assert_array_equal(cache.codes[5:6, :, i].cpu().numpy(), c)
    out = torch.empty((1, 3, 128), dtype=torch.float32, device="cuda")
    out2 = torch.empty_like(out)
    bst.kv4_load(cache, slots, out, out2)
    np.testing.assert_array_equal(_f64(out), dequantise(*quantise(_f64(x))))


def test_store_takes_no_rows():
    cache = bst.KV4Cache.empty(1, 2, 64, "cuda")
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, dtype=torch.int32, device="cuda")
    bst.kv4_store(e, e, s, cache)
    bst.kv4_load(cache, s, e, e)


# ---------------------------------------------------------------- attention

def _cache(form, kind, pages, hkv, d, seed, poison=None):
    """A cache and its float64 K and V; poison: (slots, value) written into V and K of some slots (16-bit) or their
    scales (4-bit)."""
    g = _gen(seed)
    k, v = (torch.randn((pages * 64, hkv, d), generator=g, device="cuda") *
            torch.exp(0.5 * torch.randn((1, hkv, d), generator=g, device="cuda")) for _ in range(2))
    if form == "kv16":
        pool = torch.empty((pages * 64, 2, hkv, d), dtype=TYPES[kind], device="cuda")  # K and V interleaved by slot
        pool[:, 0], pool[:, 1] = k, v
        if poison is not None:
            pool[poison[0], :] = poison[1]
        return bst.KV16Cache(pool[:, 0], pool[:, 1]), _f64(pool[:, 0]), _f64(pool[:, 1])
    c, s = [], []
    for x in (_f64(k), _f64(v)):
        a, b = quantise(x)
        c.append(a), s.append(b)
    c, s = np.stack(c, 2), np.stack(s, 2)
    if poison is not None:
        s[poison[0]] = 255
    kv = dequantise(c, s)
    return (bst.KV4Cache(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()), kv[:, :, 0], kv[:, :, 1])


def _queries(rows, hq, d, kind, seed, guard=3):
    """q inside a wider buffer, out inside a wider one with sentinels, lse."""
    g = _gen(seed)
    wide = torch.randn((rows, hq + 2, d), generator=g, device="cuda").to(TYPES[kind])
    out = torch.full((rows + guard, hq + 1, d), -77.0, dtype=TYPES[kind], device="cuda")
    lse = torch.full((rows + guard, hq), -77.0, dtype=torch.float32, device="cuda")
    return wide[:, 1:hq + 1], out, lse


def _intact(out, lse, rows, hq, left=()):
    assert (out[rows:] == -77.0).all() and (out[:, hq:] == -77.0).all() and (lse[rows:] == -77.0).all()
    for r in left:
        assert (out[r] == -77.0).all() and (lse[r] == -77.0).all(), r


SLOT_CASES = [  # kind, form, d, hq, hkv, ld, counts
    ("bf16", "kv4", 128, 16, 2, 2051, [2050, 2051, 0, 1, 31]),
    ("bf16", "kv4", 128, 1, 1, 1, [1, 0, -3]),
    ("bf16", "kv4", 128, 24, 1, 300, [32, 33, 300, 128, 129]),
    ("bf16", "kv4", 128, 40, 1, 70, [64, 65, 7]),
    ("bf16", "kv4", 64, 7, 7, 257, [256, 257, 255]),
    ("f16", "kv4", 64, 28, 4, 511, [510, 3, 511, 160]),
    ("f16", "kv4", 256, 16, 2, 190, [190, 96, 95, 2]),
    ("bf16", "kv4", 256, 20, 1, 190, [190, 96, 95, 2]),
    ("bf16", "kv16", 128, 16, 2, 515, [514, 0, 515, 129]),
    ("f16", "kv16", 128, 32, 1, 200, [200, 64, 63]),
    ("f16", "kv16", 64, 3, 3, 130, [130, 32, 17]),
    ("bf16", "kv16", 256, 8, 1, 97, [97, 96, 1]),
    ("f16", "kv16", 256, 24, 1, 97, [97, 96, 1]),
    ("bf16", "kv16", 64, 96, 2, 97, [97, 96, 1]),
]


@pytest.mark.parametrize("kind,form,d,hq,hkv,ld,counts", SLOT_CASES)
def test_slots_matches_the_definition(kind, form, d, hq, hkv, ld, counts):
    say(f"attn_slots {kind} {form} d={d} hq={hq} hkv={hkv} ld={ld} counts={counts}")
    pages = 40
    rows = len(counts)
    cache, K, V = _cache(form, kind, pages, hkv, d, 11 * d + hq)
    rng = np.random.default_rng(ld + hq)
    lists = rng.integers(0, pages * 64, size=(rows, ld)).astype(np.int32)
    lists[rng.random((rows, ld)) < 0.05] = -1                    # sentinels inside the list
    lists[rng.random((rows, ld)) < 0.02] = pages * 64 + 5        # past the pool: not read
    if rows > 1:
        lists[0, :min(ld, 40)] = -1                              # a step with no key at all
    q, out, lse = _queries(rows, hq, d, kind, 5)
    slots, cnt = torch.from_numpy(lists).cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda")
    scale = 0.11
    want, n = [], []
    for r in range(rows):
        s = lists[r, :max(0, min(counts[r], ld))]
        s = s[(s >= 0) & (s < pages * 64)]
        want.append(attend_row(_f64(q[r]), K[s], V[s], scale))
        n.append(len(s))
    ws = bst.attn_workspace("cuda")
    for workspace in (ws, None, ws):
        out.fill_(-77.0), lse.fill_(-77.0)
        bst.attn_slots(q, cache, slots, out[:rows, :hq], count=cnt, scale=scale, lse=lse[:rows], workspace=workspace)
        torch.cuda.synchronize()
        check_rows(_f64(out[:rows, :hq]), _f64(lse[:rows]), want, kind, n, np.nanmax(np.abs(V)))
        _intact(out, lse, rows, hq)
    assert not ws[:65536].any()                                  # the counters are zero again
    first = out.clone()
    for _ in range(3):                                           # bit for bit the same however the splits arrive
        bst.attn_slots(q, cache, slots, out[:rows, :hq], count=cnt, scale=scale, workspace=ws)
        assert torch.equal(out, first)


def test_slots_without_counts_reads_the_whole_list():
    cache, K, V = _cache("kv4", "bf16", 3, 2, 128, 4)
    lists = np.full((2, 150), -1, np.int32)
    lists[0, 3:90] = np.arange(87)
    q, out, lse = _queries(2, 8, 128, "bf16", 6)
    bst.attn_slots(q, cache, torch.from_numpy(lists).cuda(), out[:2, :8], lse=lse[:2])
    want = [attend_row(_f64(q[r]), K[s], V[s], 128 ** -0.5) for r, s in ((0, np.arange(87)), (1, np.arange(0)))]
    check_rows(_f64(out[:2, :8]), _f64(lse[:2]), want, "bf16", [87, 0], np.abs(V).max())
    assert (out[1, :8] == 0).all() and torch.isneginf(lse[1]).all()
    out.fill_(-77.0)
    bst.attn_slots(q, cache, torch.empty((2, 0), dtype=torch.int32, device="cuda"), out[:2, :8], lse=lse[:2],
                   workspace=bst.attn_workspace("cuda"))         # lists of no entries
    assert (out[:2, :8] == 0).all() and torch.isneginf(lse[:2]).all()
    _intact(out, lse, 2, 8)


@pytest.mark.parametrize("form", ["kv4", "kv16"])
def test_slots_takes_no_harm_from_unlisted_nan_and_passes_listed_nan(form):
    """Slot 0 stands in for missing keys inside the kernel: it and others hold
    NaN and must not be seen unless listed."""
    poison = (np.array([0, 1, 63, 64]), float("nan"))
    cache, K, V = _cache(form, "bf16", 2, 2, 128, 9, poison)
    lists = np.full((3, 70), -1, np.int32)
    lists[0, 5:60] = np.arange(2, 57)
    lists[1, :] = np.r_[np.arange(2, 62), np.arange(65, 75)]
    lists[2, :40] = np.arange(30, 70)                            # holds 63 and 64
    q, out, lse = _queries(3, 4, 128, "bf16", 8)
    bst.attn_slots(q, cache, torch.from_numpy(lists).cuda(), out[:3, :4], lse=lse[:3])
    torch.cuda.synchronize()
    want = [attend_row(_f64(q[r]), K[lists[r][lists[r] >= 0]], V[lists[r][lists[r] >= 0]], 128 ** -0.5) for r in (0, 1)]
    check_rows(_f64(out[:2, :4]), _f64(lse[:2]), want, "bf16", [55, 70], 10.0)
    assert torch.isnan(out[2, :4]).all() and torch.isnan(lse[2]).all()


def test_slots_extreme_scores():
    """Scores of thousands, all equal scores, and a lone key far below the rest."""
    d, n = 128, 200
    k = torch.randn((256, 1, d), generator=_gen(1), device="cuda") * 30
    k[100:140] = k[100]
    cache = bst.KV16Cache(k.bfloat16(), torch.randn((256, 1, d), generator=_gen(2), device="cuda").bfloat16())
    K, V = _f64(cache.k), _f64(cache.v)
    q, out, lse = _queries(3, 4, d, "bf16", 3)
    q = q.clone() * 30
    lists = np.stack([np.arange(n), np.r_[np.arange(100, 140), np.full(n - 40, -1)], np.r_[np.arange(n - 1, -1, -1)]]).astype(np.int32)
    bst.attn_slots(q, cache, torch.from_numpy(lists).cuda(), out[:3, :4], lse=lse[:3], workspace=bst.attn_workspace("cuda"))
    want = [attend_row(_f64(q[r]), K[x[x >= 0]], V[x[x >= 0]], d ** -0.5) for r, x in enumerate(lists)]
    check_rows(_f64(out[:3, :4]), _f64(lse[:3]), want, "bf16", [n, 40, n], np.abs(V).max())


@pytest.mark.parametrize("scale", [0.0, -0.3, -1e-30, 3.0])
@pytest.mark.parametrize("rows", [2, 40])
def test_any_finite_scale(scale, rows):
    say(f"scale {scale} rows={rows}")
    pt, ptr, pos, pages = _batch([200], [rows], 4)
    cache, K, V = _cache("kv4", "bf16", pages, 2, 128, 12)
    q, out, lse = _queries(rows, 8, 128, "bf16", 3)
    res, n = _window_want(_f64(q), K, V, pt, ptr, pos, pages, rows, 70, 3, scale)
    bst.attn_window(q, cache, *[torch.from_numpy(x).cuda() for x in (pt, ptr, pos)], rows, 70, 3, out[:rows, :8], scale=scale,
                    lse=lse[:rows], workspace=bst.attn_workspace("cuda"))
    check_rows(_f64(out[:rows, :8]), _f64(lse[:rows]), res, "bf16", n, np.abs(V).max())


def _batch(ctx, rows_per_req, seed, extra_rows=0, stride_extra=1):
    """page_table (random pages, -1 behind a request's), req_row_ptr, positions at the end of each context, pages."""
    rng = np.random.default_rng(seed)
    pages = [max(1, -(-t // 64)) for t in ctx]
    perm = rng.permutation(sum(pages))
    pt = np.full((len(ctx), max(pages) + stride_extra), -1, np.int32)
    at = 0
    for b, p in enumerate(pages):
        pt[b, :p] = perm[at:at + p]
        at += p
    ptr = np.concatenate([[0], np.cumsum(rows_per_req)]).astype(np.int32)
    pos = np.concatenate([np.arange(t - n, t) for t, n in zip(ctx, rows_per_req)] + [np.full(extra_rows, 3)]).astype(np.int32)
    return pt, ptr, pos, sum(pages)


def _window_want(q, K, V, pt, ptr, pos, num_pages, max_rows, window, sinks, scale):
    """Per row of a request: attend_row's results and the count of keys; None for rows that are left alone."""
    res, n = [None] * len(pos), [0] * len(pos)
    for b in range(len(ptr) - 1):
        for r in range(ptr[b], min(ptr[b + 1], ptr[b] + max_rows)):
            t = int(pos[r])
            p = np.arange(0, max(0, min(t + 1, pt.shape[1] * 64)))
            p = p[(p > t - window) | (p < sinks)]
            page = pt[b][p // 64]
            ok = (page >= 0) & (page < num_pages)
            s = page[ok].astype(np.int64) * 64 + p[ok] % 64
            res[r] = attend_row(q[r], K[s], V[s], scale)
            n[r] = len(s)
    return res, n


def _check_window(kind, form, d, hq, hkv, pt, ptr, pos, pages, max_rows, window, sinks, seed, poison=None, workspaces=None):
    cache, K, V = _cache(form, kind, pages, hkv, d, seed, poison)
    rows = len(pos)
    q, out, lse = _queries(rows, hq, d, kind, seed + 1)
    scale = 0.09
    res, n = _window_want(_f64(q), K, V, pt, ptr, pos, pages, max_rows, window, sinks, scale)
    done = [r for r in range(rows) if res[r] is not None]
    args = [torch.from_numpy(x).cuda() for x in (pt, ptr, pos)]
    for ws in workspaces or (bst.attn_workspace("cuda"), None):
        out.fill_(-77.0), lse.fill_(-77.0)
        bst.attn_window(q, cache, *args, max_rows, window, sinks, out[:rows, :hq], scale=scale, lse=lse[:rows], workspace=ws)
        torch.cuda.synchronize()
        vmax = np.max(np.abs(V[np.isfinite(V)]))
        check_rows(_f64(out[done, :hq]), _f64(lse[done]), [res[r] for r in done], kind, [n[r] for r in done], vmax)
        _intact(out, lse, rows, hq, [r for r in range(rows) if res[r] is None])


WINDOW_CASES = [  # kind, form, d, hq, hkv, contexts, rows, max_rows, window, sinks
    ("bf16", "kv4", 128, 16, 2, [1, 64, 65, 700, 300], [1, 1, 1, 1, 1], 1, 128, 4),
    ("bf16", "kv4", 128, 8, 1, [40, 500, 6, 200], [6, 6, 6, 3], 6, 100, 4),
    ("bf16", "kv16", 128, 16, 2, [40, 500, 6, 200], [6, 0, 6, 3], 6, 33, 70),
    ("f16", "kv4", 64, 6, 6, [400, 65], [5, 2], 5, 64, 0),
    ("f16", "kv16", 64, 20, 1, [130, 131], [4, 4], 4, 1, 1),
    ("f16", "kv16", 256, 8, 2, [300, 20], [2, 2], 2, 1000, 4),
    ("bf16", "kv4", 256, 4, 2, [300, 20], [2, 3], 3, 77, 5),
    ("bf16", "kv16", 128, 4, 1, [333, 64], [200, 64], 200, 90, 3),      # prefill
    ("bf16", "kv16", 128, 8, 1, [333], [333], 333, 2147483647, 0),      # plain causal
    ("bf16", "kv16", 128, 6, 2, [700, 90, 129], [257, 90, 129], 257, 200, 66),
    ("f16", "kv16", 128, 7, 1, [260, 300], [130, 131], 131, 64, 130),
    ("bf16", "kv4", 128, 8, 2, [500, 90], [300, 70], 300, 129, 4),
    ("f16", "kv4", 128, 12, 4, [260], [200], 200, 100, 13),
    ("bf16", "kv16", 64, 8, 2, [400, 33], [260, 33], 260, 150, 2),
    ("bf16", "kv4", 64, 16, 2, [400, 33], [260, 33], 260, 150, 2),
    ("bf16", "kv4", 256, 4, 2, [200], [150], 150, 80, 4),
    ("f16", "kv16", 256, 4, 4, [200], [150], 150, 80, 4),
    ("f16", "kv4", 64, 4, 1, [300], [290], 290, 70, 4),
    ("bf16", "kv16", 256, 4, 2, [200], [150], 150, 80, 4),
    ("f16", "kv4", 256, 2, 1, [200], [150], 150, 80, 4),
    ("bf16", "kv16", 128, 3, 3, [150], [140], 140, 0, 5),               # sinks only
    ("bf16", "kv16", 128, 2, 1, [150], [140], 140, 0, 0),               # nothing to see
    ("bf16", "kv4", 128, 2, 1, [70], [3], 3, 0, 0),
]


@pytest.mark.parametrize("kind,form,d,hq,hkv,ctx,rows,max_rows,window,sinks", WINDOW_CASES)
def test_window_matches_the_definition(kind, form, d, hq, hkv, ctx, rows, max_rows, window, sinks):
    say(f"attn_window {kind} {form} d={d} hq={hq} hkv={hkv} ctx={ctx} rows={rows} window={window} sinks={sinks}")
    pt, ptr, pos, pages = _batch(ctx, rows, d + hq, extra_rows=2)
    _check_window(kind, form, d, hq, hkv, pt, ptr, pos, pages, max_rows, window, sinks, 3 * d + hq)


@pytest.mark.parametrize("max_rows", [5, 200])
def test_window_odd_rows(max_rows):
    """Unsorted and repeated positions, padding rows (t < 0), positions past the
    page table, pages that hold nothing, rows past max_rows."""
    say(f"attn_window odd rows max_rows={max_rows}")
    pt, ptr, pos, pages = _batch([400, 300, 260], [7, 203, 4], 5, extra_rows=1, stride_extra=0)
    rng = np.random.default_rng(2)
    pos[:7] = [399, -1, 20, 20, 150, 5000, 0]
    pos[7:210] = rng.integers(-3, 300, 203)
    pt[0, 1], pt[1, 2], pt[2, 0] = -1, pages, 2 ** 30            # no such pages
    for form in ("kv16", "kv4"):
        _check_window("bf16", form, 128, 8, 2, pt, ptr, pos, pages, max_rows, 90, 70, 17)


@pytest.mark.parametrize("form,bad", [("kv16", float("nan")), ("kv16", float("inf")), ("kv16", -float("inf")),
                                      ("kv4", float("nan"))])  # the 4-bit cache holds no infinities
@pytest.mark.parametrize("rows", [5, 150])
def test_window_masked_infinities_and_nan(form, bad, rows):
    """Slots of positions that some rows of a tile see and others do not hold
    infinities or NaN (K and V): only the rows that see them show it."""
    say(f"attn_window masked {form} {bad} rows={rows}")
    pt, ptr, pos, pages = _batch([200], [rows], 8)
    at = np.array([pt[0, p // 64] * 64 + p % 64 for p in (198, 199, 90)])
    _check_window("bf16", form, 128, 4, 1, pt, ptr, pos, pages, rows, 60, 4, 23, poison=(at, bad))


@pytest.mark.parametrize("rows", [5, 150])
def test_window_masked_infinite_values(rows):
    """The same with finite keys: an infinity in V reaches the rows that see it
    as that infinity, both signs as NaN."""
    say(f"attn_window infinite values rows={rows}")
    pt, ptr, pos, pages = _batch([200], [rows], 8)
    cache, K, V = _cache("kv16", "bf16", pages, 1, 128, 31)
    for p, ch, x in ((199, 3, np.inf), (198, 3, -np.inf), (197, 64, np.inf), (60, 100, -np.inf), (197, 127, np.nan)):
        s = int(pt[0, p // 64]) * 64 + p % 64
        cache.v[s, 0, ch] = x
        V[s, 0, ch] = x
    q, out, lse = _queries(rows, 4, 128, "bf16", 2)
    res, n = _window_want(_f64(q), K, V, pt, ptr, pos, pages, rows, 60, 4, 0.09)
    bst.attn_window(q, cache, *[torch.from_numpy(x).cuda() for x in (pt, ptr, pos)], rows, 60, 4, out[:rows, :4], scale=0.09,
                    lse=lse[:rows], workspace=bst.attn_workspace("cuda"))
    check_rows(_f64(out[:rows, :4]), _f64(lse[:rows]), res, "bf16", n, np.max(np.abs(V[np.isfinite(V)])))


# Small batches of many rows are gathered.  What follows makes the same batches
# long enough for the prefill kernel: with requests that have no rows, or with a
# page table much wider than the contexts (whose pages the kernel then splits).

def _with_empty_requests(pt, ptr, max_rows, hq, hkv, window, sinks):
    """At least 800,000 row tiles (of 32 pairs) times keys, which the kernels' rule puts on the prefill side."""
    tiles = -(-max_rows * hq // 32)
    n = 800_000 // (tiles * min(pt.shape[1] * 64, window + sinks + 1)) + 1
    return np.concatenate([pt, np.full((n, pt.shape[1]), -1, np.int32)]), np.concatenate([ptr, np.full(n, ptr[-1], np.int32)])


@pytest.mark.parametrize("kind,form,d,hq,hkv,ctx,rows,max_rows,window,sinks",
                         [c for c in WINDOW_CASES if c[7] >= 130 and not (c[1] == "kv4" and c[2] == 256)])
def test_window_prefill_matches_the_definition(kind, form, d, hq, hkv, ctx, rows, max_rows, window, sinks):
    say(f"attn_window prefill {kind} {form} d={d} hq={hq} hkv={hkv} ctx={ctx} rows={rows} window={window} sinks={sinks}")
    pt, ptr, pos, pages = _batch(ctx, rows, d + hq, extra_rows=2)
    pt, ptr = _with_empty_requests(pt, ptr, max_rows, hq, hkv, window, sinks)
    _check_window(kind, form, d, hq, hkv, pt, ptr, pos, pages, max_rows, window, sinks, 3 * d + hq)


@pytest.mark.parametrize("kind,form,d,hq,hkv,ctx,rows", [
    ("bf16", "kv16", 128, 4, 1, [333, 64], [200, 64]), ("f16", "kv4", 128, 7, 1, [700], [150]),
    ("bf16", "kv4", 64, 16, 2, [400, 33], [260, 33]), ("f16", "kv16", 64, 8, 8, [300], [290]),
    ("bf16", "kv16", 256, 4, 2, [900, 1], [50, 1]), ("bf16", "kv4", 128, 8, 2, [1500], [170])])
@pytest.mark.parametrize("window,sinks", [(2**31 - 1, 0), (0, 1 << 30), (1 << 24, 3)])
def test_window_prefill_split_pages(kind, form, d, hq, hkv, ctx, rows, window, sinks):
    """Pages split over workgroups, most of whose parts are empty."""
    say(f"attn_window prefill split {kind} {form} d={d} hq={hq} hkv={hkv} ctx={ctx} rows={rows} window={window} sinks={sinks}")
    pt, ptr, pos, pages = _batch(ctx, rows, d + hq, extra_rows=2, stride_extra=30000)
    _check_window(kind, form, d, hq, hkv, pt, ptr, pos, pages, max(rows), window, sinks, 3 * d + hq)


def test_window_prefill_odd_rows():
    """test_window_odd_rows by the prefill kernel."""
    say("attn_window prefill odd rows")
    pt, ptr, pos, pages = _batch([400, 300, 260], [7, 203, 4], 5, extra_rows=1, stride_extra=0)
    rng = np.random.default_rng(2)
    pos[:7] = [399, -1, 20, 20, 150, 5000, 0]
    pos[7:210] = rng.integers(-3, 300, 203)
    pt[0, 1], pt[1, 2], pt[2, 0] = -1, pages, 2 ** 30            # no such pages
    pt, ptr = _with_empty_requests(pt, ptr, 200, 8, 2, 90, 70)
    for form in ("kv16", "kv4"):
        _check_window("bf16", form, 128, 8, 2, pt, ptr, pos, pages, 200, 90, 70, 17)


@pytest.mark.parametrize("form,bad", [("kv16", float("nan")), ("kv16", float("inf")), ("kv16", -float("inf")),
                                      ("kv4", float("nan"))])
@pytest.mark.parametrize("split", [False, True])
def test_window_prefill_masked_infinities_and_nan(form, bad, split):
    say(f"attn_window prefill masked {form} {bad} split={split}")
    pt, ptr, pos, pages = _batch([200], [150], 8, stride_extra=30000 if split else 1)
    window, sinks = (2**31 - 1, 0) if split else (60, 4)
    if not split:
        pt, ptr = _with_empty_requests(pt, ptr, 150, 4, 1, window, sinks)
    at = np.array([pt[0, p // 64] * 64 + p % 64 for p in (198, 199, 90)])
    _check_window("bf16", form, 128, 4, 1, pt, ptr, pos, pages, 150, window, sinks, 23, poison=(at, bad))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("split", [False, True])
def test_window_prefill_masked_infinite_values(kind, split):
    """Finite keys: an infinity in V reaches the rows that see it as that infinity, both signs as NaN."""
    say(f"attn_window prefill infinite values {kind} split={split}")
    pt, ptr, pos, pages = _batch([200], [150], 8, stride_extra=30000 if split else 1)
    window, sinks = (2**31 - 1, 0) if split else (60, 4)
    if not split:
        pt, ptr = _with_empty_requests(pt, ptr, 150, 4, 1, window, sinks)
    cache, K, V = _cache("kv16", kind, pages, 1, 128, 31)
    for p, ch, x in ((199, 3, np.inf), (198, 3, -np.inf), (197, 64, np.inf), (60, 100, -np.inf), (197, 127, np.nan)):
        s = int(pt[0, p // 64]) * 64 + p % 64
        cache.v[s, 0, ch] = x
        V[s, 0, ch] = x
    q, out, lse = _queries(150, 4, 128, kind, 2)
    res, n = _window_want(_f64(q), K, V, pt, ptr, pos, pages, 150, window, sinks, 0.09)
    bst.attn_window(q, cache, *[torch.from_numpy(x).cuda() for x in (pt, ptr, pos)], 150, window, sinks, out[:150, :4], scale=0.09,
                    lse=lse[:150], workspace=bst.attn_workspace("cuda"))
    check_rows(_f64(out[:150, :4]), _f64(lse[:150]), res, kind, n, np.max(np.abs(V[np.isfinite(V)])))


def test_long_split_lists_join_in_rounds():
    """Rows of few heads and many, whose parts are joined 16, 8 and 4 at a time (one part's columns short of its tile's)."""
    for hq, hkv, d, k in ((28, 1, 128, 600), (28, 1, 128, 2100), (13, 1, 256, 2100), (5, 1, 64, 9000), (28, 1, 128, 40000),
                          (16, 1, 256, 40000)):
        say(f"attn_slots split hq={hq} d={d} k={k}")
        cache, K, V = _cache("kv4", "bf16", 40, hkv, d, 3)
        rng = np.random.default_rng(k)
        lists = rng.integers(0, 2560, (2, k)).astype(np.int32)
        lists[1, ::3] = -1
        q, out, lse = _queries(2, hq, d, "bf16", 5)
        want = [attend_row(_f64(q[r]), K[x[x >= 0]], V[x[x >= 0]], d ** -0.5) for r, x in enumerate(lists)]
        bst.attn_slots(q, cache, torch.from_numpy(lists).cuda(), out[:2, :hq], lse=lse[:2], workspace=bst.attn_workspace("cuda"))
        torch.cuda.synchronize()
        check_rows(_f64(out[:2, :hq]), _f64(lse[:2]), want, "bf16", [k, k - -(-k // 3)], np.abs(V).max())


@pytest.mark.parametrize("form", ["kv4", "kv16"])
def test_pools_past_4_gib(form):
    """Slots whose byte offsets pass 32 bits."""
    say(f"pool past 4 GiB {form}")
    hkv, d = 8, 128
    slots_total = (1 << 32) // (hkv * d * (1 if form == "kv4" else 2)) + 64 * 1000
    pages = slots_total // 64
    near = torch.arange(40, device="cuda")
    far = pages * 64 - 1 - torch.arange(200, device="cuda")
    lists = torch.cat([far, near]).int()
    k, v = (torch.randn((240, hkv, d), generator=_gen(i), device="cuda").bfloat16() for i in (1, 2))
    if form == "kv4":
        cache = bst.KV4Cache.empty(pages, hkv, d, "cuda")
        bst.kv4_store(k, v, lists, cache)
        K, V = (dequantise(*quantise(_f64(x))) for x in (k, v))
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        bst.kv4_load(cache, lists, ko, vo)
        np.testing.assert_array_equal(_f64(ko), K), np.testing.assert_array_equal(_f64(vo), V)
    else:
        pools = [torch.zeros((pages * 64, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for p, x in zip(pools, (k, v)):
            p[lists.long()] = x
        cache, K, V = bst.KV16Cache(*pools), _f64(k), _f64(v)
    q, out, lse = _queries(1, 16, d, "bf16", 4)
    bst.attn_slots(q, cache, lists.view(1, -1), out[:1, :16], lse=lse[:1])
    want = attend_row(_f64(q[0]), K, V, d ** -0.5)
    check_rows(_f64(out[:1, :16]), _f64(lse[:1]), [want], "bf16", [240], np.abs(V).max())
    # the same keys as positions of a request: whole pages at the far end
    page = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    order = (page[0].long()[:, None] * 64 + torch.arange(64, device="cuda")).flatten()[:150]
    if form == "kv4":
        ko, vo = torch.empty((150, hkv, d), dtype=torch.float32, device="cuda"), torch.empty((150, hkv, d), dtype=torch.float32, device="cuda")
        bst.kv4_load(cache, order.int(), ko, vo)
    else:
        ko, vo = cache.k[order], cache.v[order]
    K, V = _f64(ko), _f64(vo)
    for rows in (1, 150):
        q, out, lse = _queries(rows, 16, d, "bf16", 4)
        pos = torch.arange(150 - rows, 150, dtype=torch.int32, device="cuda")
        ptr = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        bst.attn_window(q, cache, page, ptr, pos, rows, 1000, 0, out[:rows, :16], lse=lse[:rows], workspace=bst.attn_workspace("cuda"))
        some = [0, rows // 2, rows - 1]
        want = [attend_row(_f64(q[r]), K[:int(pos[r]) + 1], V[:int(pos[r]) + 1], d ** -0.5) for r in some]
        check_rows(_f64(out[some, :16]), _f64(lse[some]), want, "bf16", [150] * 3, np.abs(V).max())
    del cache
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- as they are used

def test_the_path_from_store_to_attention():
    """Raw keys compressed, rows scored and selected, K/V stored in 4 bits, and
    the chosen slots attended, on a stream of its own: against the reference
    over the slots that the selection wrote."""
    import synth
    from block_scoring_top_amd.pipeline import IndexerPath
    from synth.device import upload
    inp = synth.qsa_verify_64req(B=4, lo=300, hi=9000)
    say(f"path rows={inp.num_rows} k={inp.k}")
    dev = upload(inp, "cuda")
    hkv, hq, d = 2, 16, 128
    pages = inp.num_pages
    n = pages * 64
    k, v = (torch.randn((n, hkv, d), generator=_gen(i), device="cuda").bfloat16() for i in (5, 6))
    q, out, lse = _queries(inp.num_rows, hq, d, "bf16", 7)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        cache = bst.KV4Cache.empty(pages, hkv, d, "cuda")
        every = torch.arange(n, dtype=torch.int32, device="cuda")
        bst.kv4_store(k, v, every, cache)
        p = IndexerPath(dev, "decode")
        p.run()
        p.attend(q, cache, out[:inp.num_rows, :hq], lse=lse[:inp.num_rows])
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        bst.kv4_load(cache, every, ko, vo)
    s.synchronize()
    K, V = _f64(ko), _f64(vo)
    np.testing.assert_array_equal(K, dequantise(*quantise(_f64(k))))
    slots, cnt = p.slots.cpu().numpy(), p.out_count.cpu().numpy()
    want, m = [], []
    for r in range(inp.num_rows):
        x = slots[r, :cnt[r]]
        x = x[x >= 0]
        want.append(attend_row(_f64(q[r]), K[x], V[x], d ** -0.5))
        m.append(len(x))
    assert min(m) > 0
    check_rows(_f64(out[:inp.num_rows, :hq]), _f64(lse[:inp.num_rows]), want, "bf16", m, np.abs(V).max())


def test_the_path_attends_first_on_another_stream(monkeypatch):
    """The path's attention workspace is made by the first attend(): cleared on
    the stream that the call goes to, while the current stream is still busy
    and the memory at hand is dirty; refused while that stream captures."""
    import synth
    from block_scoring_top_amd.pipeline import IndexerPath
    from synth.device import upload
    inp = synth.qsa_verify_64req(B=2, lo=300, hi=3000)
    say(f"attend first on another stream, rows={inp.num_rows}")
    dev = upload(inp, "cuda")
    cache, _, _ = _cache("kv4", "bf16", inp.num_pages, 2, 128, 11)
    q, want, _ = _queries(inp.num_rows, 16, 128, "bf16", 12)
    p = IndexerPath(dev, "decode")
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        with pytest.raises(RuntimeError, match="captured"):
            p.attend(q, cache, want[:inp.num_rows, :16])
    assert p.attn_ws is None
    p.run()
    p.attend(q, cache, want[:inp.num_rows, :16])
    got = torch.full_like(want, -77.0)
    p.attn_ws = None
    dirty = torch.full((bst.ATTN_WORKSPACE_BYTES,), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    del dirty
    x = torch.randn((4096, 4096), device="cuda")
    for _ in range(20):  # keeps the current stream busy for some ms
        x = x @ x * 1e-3
    p.attend(q, cache, got[:inp.num_rows, :16], stream=s)
    s.synchronize()
    assert torch.equal(got[:inp.num_rows, :16], want[:inp.num_rows, :16])
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows", [[1, 1, 1], [150, 70, 2]])
def test_bounds_past_32_bits_mean_no_bound(rows):
    """window, sinks and max_rows larger than any position or row count."""
    ctx = [700, 130, 2]
    pt, ptr, pos, pages = _batch(ctx, rows, 31)
    say(f"bounds past 32 bits, rows={rows}")
    cache, _, V = _cache("kv16", "bf16", pages, 2, 128, 32)
    q, _, _ = _queries(len(pos), 8, 128, "bf16", 33)
    args = [torch.from_numpy(x).cuda() for x in (pt, ptr, pos)]
    ws = bst.attn_workspace("cuda")
    outs = []
    for max_rows, window, sinks in ((max(rows), 2**31 - 1, 0), (1 << 40, 1 << 32, 0), (2**31 - 1, 0, 1 << 33)):
        out = torch.full((len(pos), 8, 128), -77.0, dtype=torch.bfloat16, device="cuda")
        bst.attn_window(q, cache, *args, max_rows, window, sinks, out, workspace=ws)
        outs.append(out)
    torch.cuda.synchronize()
    # The calls may take different kernels.  In each, the weights and their sum
    # are rounded by at most 2^-8 of the result, and so is the output.
    for o in outs[1:]:
        assert (o.float() - outs[0].float()).abs().max().item() <= 2 * 3 * 2**-8 * np.abs(V).max()


@pytest.mark.parametrize("case", ["slots", "window_decode", "window_prefill", "store"])
def test_captured_calls_replay_like_eager(case):
    """Captured once, replayed with new inputs between eager work, each replay
    bit for bit like the eager call."""
    say(f"graph {case}")
    hkv, hq, d = 2, 16, 128
    pt, ptr, pos, pages = _batch([700, 260], [1, 1] if case != "window_prefill" else [300, 200], 3)
    rows = len(pos)
    cache, _, _ = _cache("kv4", "bf16", pages, hkv, d, 5)
    ws = bst.attn_workspace("cuda")
    q = torch.empty((rows, hq, d), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((rows, hq), dtype=torch.float32, device="cuda")
    lists = torch.randint(-1, pages * 64, (rows, 700), generator=_gen(1), device="cuda", dtype=torch.int32)
    at = torch.arange(100, 100 + rows, dtype=torch.int32, device="cuda")
    meta = [torch.from_numpy(x).cuda() for x in (pt, ptr, pos)]
    kin = torch.empty((rows, hkv, d), dtype=torch.bfloat16, device="cuda")
    ko, vo = torch.empty_like(kin), torch.empty_like(kin)

    def call():
        if case == "slots":
            bst.attn_slots(q, cache, lists, out, lse=lse, workspace=ws)
        elif case == "store":
            bst.kv4_store(kin, kin, at, cache)
            bst.kv4_load(cache, at, ko, vo)
        else:
            bst.attn_window(q, cache, *meta, 1 if case == "window_decode" else 300, 150, 4, out, lse=lse, workspace=ws)

    def fill(i):
        q.copy_(torch.randn(q.shape, generator=_gen(50 + i), device="cuda"))
        kin.copy_(torch.randn(kin.shape, generator=_gen(90 + i), device="cuda"))

    result = lambda: [x.clone() for x in ((ko, vo) if case == "store" else (out, lse))]  # noqa: E731
    want = []
    for i in range(3):
        fill(i)
        call()
        torch.cuda.synchronize()
        want.append(result())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    torch.cuda.synchronize()
    for rep in range(2):
        for i in range(3):
            fill(i)
            out.fill_(5), lse.fill_(5), ko.fill_(5), vo.fill_(5)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(result(), want[i]):
                assert torch.equal(a, b), (rep, i)


def test_two_streams_with_workspaces_of_their_own():
    """Split calls on two streams at once, each with its own workspace."""
    cache, _, _ = _cache("kv4", "bf16", 60, 2, 128, 5)
    lists = torch.randint(0, 60 * 64, (2, 3000), generator=_gen(1), device="cuda", dtype=torch.int32)
    qs = [_queries(1, 16, 128, "bf16", 20 + i)[0].clone() for i in range(2)]
    want = []
    for i in range(2):
        o = torch.empty_like(qs[i])
        bst.attn_slots(qs[i], cache, lists[i:i + 1], o, workspace=bst.attn_workspace("cuda"))
        want.append(o)
    streams, wss = [torch.cuda.Stream() for _ in range(2)], [bst.attn_workspace("cuda") for _ in range(2)]
    outs = [[torch.empty_like(qs[i]) for _ in range(20)] for i in range(2)]
    torch.cuda.synchronize()
    for k in range(20):
        for i in range(2):
            bst.attn_slots(qs[i], cache, lists[i:i + 1], outs[i][k], workspace=wss[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, want[i])


def test_prepared_and_bound_calls():
    cache, _, _ = _cache("kv4", "bf16", 4, 2, 128, 5)
    q, out, lse = _queries(3, 8, 128, "bf16", 1)
    lists = torch.randint(0, 256, (3, 99), generator=_gen(1), device="cuda", dtype=torch.int32)
    bst.attn_slots(q, cache, lists, out[:3, :8])
    want = out.clone()
    call = bst.prepare_attn_slots(q, cache, lists, out[:3, :8])
    for f in (call, call.bind()):
        out[:3, :8] = 0
        f()
        assert torch.equal(out, want)
