"""The 8-bit cache and the attention over it on the GPU, against the references
of more_ref.py and attn_ref.py (bounds derived there): codes and scales exact;
types, head layouts, page runs and paddings, appended tokens and raised scales,
special values, masks over NaN, pools past 4 GiB, graphs."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scoring_top_amd as bst
from attn_ref import attend_row, check_rows
from gpu_util import say
from more_ref import Kv8, e4m3_round, e4m3_value

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def _exps(cache):
    s = _f64(cache.scales)
    m, e = np.frexp(s)
    assert (m == 0.5).all()                                      # powers of two
    return e.astype(np.int64) - 1


def _same(cache, ref):
    np.testing.assert_array_equal(_exps(cache), ref.exps)
    got = cache.codes.cpu().numpy()
    nan = ref.codes & 127 == 127
    np.testing.assert_array_equal(got & 127 == 127, nan)
    np.testing.assert_array_equal(np.where(nan, 0, got), np.where(nan, 0, ref.codes))


def _pair(pages, hkv, d, seed, zeros=False):
    """The same cache on both sides, holding something already."""
    rng = np.random.default_rng(seed)
    codes = np.zeros((pages * 64, hkv, 2, d), np.uint8) if zeros else rng.integers(0, 256, (pages * 64, hkv, 2, d)).astype(np.uint8)
    exps = np.full((pages, hkv, 2), -120) if zeros else rng.integers(-12, 4, (pages, hkv, 2))
    cache = bst.KV8Cache(torch.from_numpy(codes).cuda(), torch.tensor(np.ldexp(1.0, exps), dtype=torch.float32, device="cuda"))
    return cache, Kv8(pages, hkv, d, codes, exps)


def _rows(T, hkv, d, kind, seed, fused):
    g = _gen(seed)
    x = torch.randn((T, 3 * hkv, d), generator=g, device="cuda") * torch.exp(1.5 * torch.randn((T, 3 * hkv, 1), generator=g, device="cuda"))
    x = x.to(TYPES[kind])
    if fused:
        return x[:, hkv:2 * hkv], x[:, 2 * hkv:]
    return x[:, hkv:2 * hkv].contiguous(), x[:, 2 * hkv:].contiguous()


def _runs(T, layout, rng):
    """Slots of T rows, those of a page within 64 rows, and the pages."""
    if layout == "chunk":                                        # one request's tokens from inside a page on
        start = int(rng.integers(0, 64))
        pages = -(-(start + T) // 64)
        perm = rng.permutation(pages + 2)
        p = np.arange(start, start + T)
        return perm[p // 64] * 64 + p % 64, pages + 2
    if layout == "decode":                                       # a page each
        perm = rng.permutation(T + 1)[:T]
        return perm * 64 + rng.integers(0, 64, T), T + 1
    # "mixed": pieces of up to 64 rows, each of some slots of one page in any order, and padding between them and inside
    slots, page = [], 0
    while len(slots) < T:
        n = int(rng.integers(1, 65))
        part = page * 64 + rng.permutation(64)[:max(1, n - n // 4)]
        part = np.concatenate([part, np.full(n - len(part), -1)])
        slots += list(rng.permutation(part))
        page += 1
    slots = np.array(slots[:T])
    order = rng.permutation(page)
    return np.where(slots >= 0, order[np.maximum(slots, 0) // 64] * 64 + slots % 64, -1), page


STORE_CASES = [  # T, hkv, d, kind, layout, fused
    (1, 1, 64, "bf16", "chunk", False), (1, 8, 256, "f32", "decode", True), (2, 3, 128, "f16", "chunk", True),
    (63, 2, 128, "bf16", "chunk", True), (64, 1, 64, "f32", "chunk", False), (65, 5, 64, "f16", "mixed", True),
    (300, 2, 128, "bf16", "mixed", False), (300, 1, 256, "f16", "mixed", True), (64, 2, 128, "bf16", "decode", True),
    (777, 3, 64, "bf16", "mixed", False), (2047, 1, 128, "f32", "chunk", False), (2048, 2, 128, "bf16", "chunk", True),
    (2500, 1, 64, "f16", "mixed", False), (2111, 3, 64, "bf16", "decode", False), (4100, 1, 256, "f32", "mixed", True),
    (5000, 1, 128, "bf16", "mixed", False)]


@pytest.mark.parametrize("T,hkv,d,kind,layout,fused", STORE_CASES)
def test_store_and_load_match_the_definition(T, hkv, d, kind, layout, fused):
    say(f"kv8 T={T} hkv={hkv} d={d} {kind} {layout} fused={fused}")
    rng = np.random.default_rng(T + d)
    slots, pages = _runs(T, layout, rng)
    if T > 10:
        slots[T // 2] = pages * 64                               # past the pool: skipped
    cache, ref = _pair(pages, hkv, d, T)
    k, v = _rows(T, hkv, d, kind, T * 7 + hkv, fused)
    bst.kv8_store(k, v, _i32(slots), cache)
    torch.cuda.synchronize()
    ref.store(_f64(k), _f64(v), slots)
    # what the other slots of a page begun anew hold is unspecified
    begun = np.zeros(pages, bool)
    there = slots[(slots >= 0) & (slots < pages * 64)]
    begun[there[there % 64 == 0] // 64] = True
    loose = np.repeat(begun, 64)
    loose[there] = False
    codes = cache.codes.cpu().numpy()
    ref.codes[loose] = codes[loose]
    _same(cache, ref)
    K, V = ref.values()
    rd = np.concatenate([rng.permutation(pages * 64)[:400], slots[:1], [-1, pages * 64, -2**31]])
    for out_kind in ("bf16", "f16", "f32"):
        out = torch.full((len(rd), 2 * hkv + 1, d), 7.0, dtype=TYPES[out_kind], device="cuda")
        bst.kv8_load(cache, _i32(rd), out[:, :hkv], out[:, hkv:2 * hkv])
        torch.cuda.synchronize()
        ok = (rd >= 0) & (rd < pages * 64)
        for x, o in ((K, out[:, :hkv]), (V, out[:, hkv:2 * hkv])):
            want = np.zeros((len(rd), hkv, d))
            want[ok] = x[rd[ok]]
            np.testing.assert_array_equal(_f64(o), _f64(torch.from_numpy(want).to(TYPES[out_kind])))
        assert (out[:, 2 * hkv:] == 7.0).all()


@pytest.mark.parametrize("T,hkv,d,kind", [(70, 2, 64, "bf16"), (150, 1, 128, "f16"), (1023, 1, 256, "bf16"), (1024, 2, 64, "f32"),
                                          (1500, 3, 128, "bf16"), (2600, 1, 256, "f16"), (1100, 2, 256, "f32")])
@pytest.mark.parametrize("per", [2, 7, 24])
@pytest.mark.parametrize("special", [False, True])
def test_store_of_interwoven_pages(T, hkv, d, kind, per, special):
    """Stretches of 64 rows, the first one shorter, each of the rows of `per` pages and padding in random order: runs of one
    to some dozens of rows that cross the kernels' groups, into pages that hold something, whose scales some outgrow."""
    say(f"kv8 woven T={T} hkv={hkv} d={d} {kind} per={per} special={special}")
    rng = np.random.default_rng(T + per)
    slots, page = [], 0
    while len(slots) < T:
        n = 64 if slots else 37
        of = rng.integers(0, per + 1, n)                         # `per`: padding
        part = np.full(n, -1)
        for q in range(per):
            at = np.nonzero(of == q)[0]
            part[at] = (page + q) * 64 + rng.permutation(np.arange(int(rng.integers(0, 2)), 64))[:len(at)]
        slots += list(part)
        page += per
    slots = np.array(slots[:T])
    order = rng.permutation(page)
    slots = np.where(slots >= 0, order[np.maximum(slots, 0) // 64] * 64 + slots % 64, -1)
    cache, ref = _pair(page, hkv, d, T)
    k, v = (x.clone() for x in _rows(T, hkv, d, kind, T * 3 + per, False))
    if special:
        for x, seed in ((k, 1), (v, 2)):
            hit = torch.rand(x.shape, generator=_gen(seed), device="cuda") < 0.003
            x[hit] = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(x.dtype).repeat(x.numel())[:int(hit.sum())]
    bst.kv8_store(k, v, _i32(slots), cache)
    torch.cuda.synchronize()
    old = ref.exps.copy()
    ref.store(_f64(k), _f64(v), slots)
    assert (ref.exps > old).any()
    begun = np.zeros(page, bool)
    there = slots[slots >= 0]
    begun[there[there % 64 == 0] // 64] = True
    loose = np.repeat(begun, 64)
    loose[there] = False
    codes = cache.codes.cpu().numpy()
    ref.codes[loose] = codes[loose]
    _same(cache, ref)


@pytest.mark.parametrize("d,kind", [(64, "f32"), (128, "bf16"), (256, "f16")])
def test_appended_tokens_raise_the_scale(d, kind):
    """Token after token into the pages of 5 requests, some larger than all before: after each call, codes and scales of
    the whole cache; then the same pages begun anew with small values."""
    say(f"kv8 append d={d} {kind}")
    rng = np.random.default_rng(d)
    cache, ref = _pair(10, 2, d, d, zeros=True)
    pages = rng.permutation(10).reshape(5, 2)
    pos = np.array([0, 60, 33, 63, 10])
    for step in range(70):
        n = 1 if step % 7 else 6
        p = pos[:, None] + np.arange(n)
        slots = (np.take_along_axis(pages, p // 64, 1) * 64 + p % 64).ravel()
        k, v = (x * 2.0 ** float(rng.integers(-6, 7)) for x in _rows(5 * n, 2, d, kind, step, step % 2))
        before = ref.exps.copy()
        bst.kv8_store(k, v, _i32(slots), cache)
        torch.cuda.synchronize()
        ref.store(_f64(k), _f64(v), slots)
        written = np.zeros(640, bool)
        for r in range(5):                                       # only what has been written since its page was begun
            for q in range(pos[r] // 64 * 64 if pos[r] // 64 else (0 if step else pos[r]), pos[r] + n):
                written[pages[r, q // 64] * 64 + q % 64] = True
        codes = cache.codes.cpu().numpy()
        ref.codes[~written] = codes[~written]
        _same(cache, ref)
        assert step < 3 or (ref.exps >= before).all() or (slots % 64 == 0).any()
        pos = (pos + n) % 120
    assert (_exps(cache) > -20).any()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_store_special_values(kind):
    """Zeros, subnormals, the ends of the range, halfway values, infinities and NaN: a head each."""
    t = TYPES[kind]
    f = torch.finfo(t)
    half = torch.tensor([448.0, 1.0625, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -10, 440.0, 432.0, 0.0, -0.0, 18.0, 17.0])
    rows = [torch.zeros(64), -torch.zeros(64), torch.full((64,), f.smallest_normal / 4), torch.full((64,), f.max),
            torch.cat([torch.full((1,), f.max), torch.full((63,), 1.0)]), torch.nn.functional.pad(half, (0, 64 - len(half))),
            torch.nn.functional.pad(half * 2.0 ** 5, (0, 64 - len(half))), torch.full((64,), float("nan"))]
    for bad in (float("inf"), -float("inf"), float("nan")):
        r = torch.linspace(-3, 3, 64)
        r[17] = bad
        rows.append(r)
    x = torch.stack(rows).to(t)[None].cuda()                     # 1 token, 11 heads
    cache, ref = _pair(1, x.shape[1], 64, 1, zeros=True)
    for slot in (5, 0):                                          # appended, and begun anew
        bst.kv8_store(x, -x, _i32([slot]), cache)
        torch.cuda.synchronize()
        ref.store(_f64(x), _f64(-x), np.array([slot]))
        ref.codes[1:] = cache.codes.cpu().numpy()[1:] if slot == 0 else ref.codes[1:]
        _same(cache, ref)
    out = [torch.empty((1, x.shape[1], 64), dtype=torch.float32, device="cuda") for _ in range(2)]
    bst.kv8_load(cache, _i32([0]), *out)
    for o, w in zip(out, ref.values()):
        np.testing.assert_array_equal(_f64(o)[0], w[0])


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_every_code_at_every_scale(kind):
    """kv8_load of all 256 codes under every scale: one rounding to the type, which only fp16 needs."""
    say(f"kv8 every code {kind}")
    e = np.arange(-120, 120)
    codes = np.tile(np.arange(256, dtype=np.uint8), (len(e) * 64, 1, 2, 1))
    cache = bst.KV8Cache(torch.from_numpy(codes).cuda(), torch.tensor(np.ldexp(1.0, e), dtype=torch.float32, device="cuda")[:, None, None].repeat(1, 1, 2).contiguous())
    out = [torch.empty((len(e), 1, 256), dtype=TYPES[kind], device="cuda") for _ in range(2)]
    bst.kv8_load(cache, _i32(np.arange(len(e)) * 64 + 7), *out)
    want = torch.from_numpy(e4m3_value(np.arange(256))[None] * np.ldexp(1.0, e)[:, None]).to(TYPES[kind])
    for o in out:
        np.testing.assert_array_equal(_f64(o[:, 0]), _f64(want))


def test_store_takes_no_rows():
    cache = bst.KV8Cache.empty(1, 2, 64, "cuda")
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, dtype=torch.int32, device="cuda")
    bst.kv8_store(e, e, s, cache)
    bst.kv8_load(cache, s, e, e)
    one = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    bst.kv8_store(one, one, _i32([-1]), cache)
    torch.cuda.synchronize()
    assert not cache.codes.any() and (cache.scales == 2.0 ** -120).all()


def test_codes_as_a_float8_tensor():
    """The cache's codes may be a float8_e4m3fn tensor: torch reads the same values."""
    cache = bst.KV8Cache(torch.zeros((128, 2, 2, 64), dtype=torch.float8_e4m3fn, device="cuda"),
                         torch.full((2, 2, 2), 2.0 ** -120, device="cuda"))
    k, v = _rows(100, 2, 64, "bf16", 3, True)
    slots = torch.arange(100, dtype=torch.int32, device="cuda")
    bst.kv8_store(k, v, slots, cache)
    ko, vo = torch.empty_like(k.contiguous()), torch.empty_like(v.contiguous())
    bst.kv8_load(cache, slots, ko, vo)
    x = cache.codes[:100].float() * cache.scales.repeat_interleave(64, 0)[:100, ..., None]
    assert torch.equal(x[:, :, 0], ko.float()) and torch.equal(x[:, :, 1], vo.float())
    # nearest codes under the page's scale: off by at most half a step, 2^-4 of the value, or 2^-10 below its normal range
    err, s = (ko.float() - k.float()).abs(), cache.scales.repeat_interleave(64, 0)[:100, :, :1]
    assert (err <= torch.maximum(2.0 ** -4 * k.float().abs(), 2.0 ** -10 * s)).all()


# ---------------------------------------------------------------- attention

def _cache(pages, hkv, d, seed, poison=None, exps=None):
    """A cache and its float64 K and V; poison: slots whose codes are all NaN."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((pages * 64, hkv, 2, d)) * np.exp(0.5 * rng.standard_normal((1, hkv, 2, d))) * 40
    codes = e4m3_round(np.clip(x, -448, 448))
    if poison is not None:
        codes[poison] = 127
    exps = rng.integers(-7, -3, (pages, hkv, 2)) if exps is None else np.broadcast_to(exps, (pages, hkv, 2))
    cache = bst.KV8Cache(torch.from_numpy(codes).cuda(), torch.tensor(np.ldexp(1.0, exps), dtype=torch.float32, device="cuda"))
    return cache, *Kv8(pages, hkv, d, codes, np.asarray(exps)).values()


def _queries(rows, hq, d, kind, seed, guard=3):
    g = _gen(seed)
    wide = torch.randn((rows, hq + 2, d), generator=g, device="cuda").to(TYPES[kind])
    out = torch.full((rows + guard, hq + 1, d), -77.0, dtype=TYPES[kind], device="cuda")
    lse = torch.full((rows + guard, hq), -77.0, dtype=torch.float32, device="cuda")
    return wide[:, 1:hq + 1], out, lse


def _intact(out, lse, rows, hq, left=()):
    assert (out[rows:] == -77.0).all() and (out[:, hq:] == -77.0).all() and (lse[rows:] == -77.0).all()
    for r in left:
        assert (out[r] == -77.0).all() and (lse[r] == -77.0).all(), r


SLOT_CASES = [  # kind, d, hq, hkv, ld, counts
    ("bf16", 128, 16, 2, 2051, [2050, 2051, 0, 1, 31]), ("bf16", 128, 1, 1, 1, [1, 0, -3]),
    ("bf16", 128, 24, 1, 300, [32, 33, 300, 128, 129]), ("f16", 128, 40, 1, 70, [64, 65, 7]),
    ("bf16", 64, 7, 7, 257, [256, 257, 255]), ("f16", 64, 28, 4, 511, [510, 3, 511, 160]),
    ("bf16", 64, 96, 2, 97, [97, 96, 1]), ("f16", 256, 16, 2, 190, [190, 96, 95, 2]), ("bf16", 256, 20, 1, 190, [190, 96, 95, 2]),
    ("f16", 128, 32, 1, 2200, [2200] * 70), ("bf16", 128, 8, 8, 64, [64, 63] * 40)]


@pytest.mark.parametrize("kind,d,hq,hkv,ld,counts", SLOT_CASES)
def test_slots_matches_the_definition(kind, d, hq, hkv, ld, counts):
    say(f"attn_slots kv8 {kind} d={d} hq={hq} hkv={hkv} ld={ld} rows={len(counts)}")
    pages, rows = 41, len(counts)
    cache, K, V = _cache(pages, hkv, d, 11 * d + hq)
    rng = np.random.default_rng(ld + hq)
    lists = rng.integers(0, pages * 64, size=(rows, ld)).astype(np.int32)
    lists[rng.random((rows, ld)) < 0.05] = -1
    lists[rng.random((rows, ld)) < 0.02] = pages * 64 + 5        # past the pool: not read
    if rows > 1:
        lists[0, :min(ld, 40)] = -1
    q, out, lse = _queries(rows, hq, d, kind, 5)
    slots, cnt = _i32(lists), _i32(counts)
    want, n = [], []
    for r in range(rows):
        s = lists[r, :max(0, min(counts[r], ld))]
        s = s[(s >= 0) & (s < pages * 64)]
        want.append(attend_row(_f64(q[r]), K[s], V[s], 0.11))
        n.append(len(s))
    ws = bst.attn_workspace("cuda")
    for workspace in (ws, None, ws):
        out.fill_(-77.0), lse.fill_(-77.0)
        bst.attn_slots(q, cache, slots, out[:rows, :hq], count=cnt, scale=0.11, lse=lse[:rows], workspace=workspace)
        torch.cuda.synchronize()
        check_rows(_f64(out[:rows, :hq]), _f64(lse[:rows]), want, kind, n, np.abs(V).max())
        _intact(out, lse, rows, hq)
    assert not ws[:65536].any()
    first = out.clone()
    for _ in range(3):
        bst.attn_slots(q, cache, slots, out[:rows, :hq], count=cnt, scale=0.11, workspace=ws)
        assert torch.equal(out, first)


def test_slots_takes_no_harm_from_unlisted_nan_and_passes_listed_nan():
    cache, K, V = _cache(2, 2, 128, 9, np.array([0, 1, 63, 64]))
    lists = np.full((3, 70), -1, np.int32)
    lists[0, 5:60] = np.arange(2, 57)
    lists[1, :] = np.r_[np.arange(2, 62), np.arange(65, 75)]
    lists[2, :40] = np.arange(30, 70)                            # holds 63 and 64
    q, out, lse = _queries(3, 4, 128, "bf16", 8)
    bst.attn_slots(q, cache, _i32(lists), out[:3, :4], lse=lse[:3])
    torch.cuda.synchronize()
    want = [attend_row(_f64(q[r]), K[lists[r][lists[r] >= 0]], V[lists[r][lists[r] >= 0]], 128 ** -0.5) for r in (0, 1)]
    check_rows(_f64(out[:2, :4]), _f64(lse[:2]), want, "bf16", [55, 70], 10.0)
    assert torch.isnan(out[2, :4]).all() and torch.isnan(lse[2]).all()


def _batch(ctx, rows_per_req, seed, extra_rows=0, stride_extra=1):
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


def _check_window(kind, d, hq, hkv, pt, ptr, pos, pages, max_rows, window, sinks, seed, poison=None):
    cache, K, V = _cache(pages, hkv, d, seed, poison)
    rows = len(pos)
    q, out, lse = _queries(rows, hq, d, kind, seed + 1)
    res, n = _window_want(_f64(q), K, V, pt, ptr, pos, pages, max_rows, window, sinks, 0.09)
    done = [r for r in range(rows) if res[r] is not None]
    args = [torch.from_numpy(x).cuda() for x in (pt, ptr, pos)]
    for ws in (bst.attn_workspace("cuda"), None):
        out.fill_(-77.0), lse.fill_(-77.0)
        bst.attn_window(q, cache, *args, max_rows, window, sinks, out[:rows, :hq], scale=0.09, lse=lse[:rows], workspace=ws)
        torch.cuda.synchronize()
        check_rows(_f64(out[done, :hq]), _f64(lse[done]), [res[r] for r in done], kind, [n[r] for r in done],
                   np.max(np.abs(V[np.isfinite(V)])))
        _intact(out, lse, rows, hq, [r for r in range(rows) if res[r] is None])


WINDOW_CASES = [  # kind, d, hq, hkv, contexts, rows, max_rows, window, sinks
    ("bf16", 128, 16, 2, [1, 64, 65, 700, 300], [1, 1, 1, 1, 1], 1, 128, 4),
    ("bf16", 128, 8, 1, [40, 500, 6, 200], [6, 6, 6, 3], 6, 100, 4),
    ("f16", 128, 16, 2, [40, 500, 6, 200], [6, 0, 6, 3], 6, 33, 70),
    ("f16", 64, 6, 6, [400, 65], [5, 2], 5, 64, 0),
    ("bf16", 64, 20, 1, [130, 131], [4, 4], 4, 1, 1),
    ("bf16", 256, 4, 2, [300, 20], [2, 3], 3, 77, 5),
    ("bf16", 128, 4, 1, [333, 64], [200, 64], 200, 90, 3),
    ("bf16", 128, 8, 1, [333], [333], 333, 2147483647, 0),
    ("f16", 128, 7, 1, [260, 300], [130, 131], 131, 64, 130),
    ("bf16", 128, 8, 2, [500, 90], [300, 70], 300, 129, 4),
    ("bf16", 64, 16, 2, [400, 33], [260, 33], 260, 150, 2),
    ("f16", 64, 4, 1, [300], [290], 290, 70, 4),
    ("f16", 256, 4, 2, [200], [150], 150, 80, 4),
    ("bf16", 128, 3, 3, [150], [140], 140, 0, 5),
    ("bf16", 128, 2, 1, [150], [140], 140, 0, 0)]


@pytest.mark.parametrize("kind,d,hq,hkv,ctx,rows,max_rows,window,sinks", WINDOW_CASES)
def test_window_matches_the_definition(kind, d, hq, hkv, ctx, rows, max_rows, window, sinks):
    say(f"attn_window kv8 {kind} d={d} hq={hq} hkv={hkv} ctx={ctx} rows={rows} window={window} sinks={sinks}")
    pt, ptr, pos, pages = _batch(ctx, rows, d + hq, extra_rows=2)
    _check_window(kind, d, hq, hkv, pt, ptr, pos, pages, max_rows, window, sinks, 3 * d + hq)


def _with_empty_requests(pt, ptr, max_rows, hq, hkv, window, sinks):
    """The same batch with enough row tiles (of 32 pairs) times keys that the kernels' rule puts it on the prefill side."""
    tiles = -(-max_rows * hq // 32)
    n = 1_600_000 // (tiles * min(pt.shape[1] * 64, window + sinks + 1)) + 1
    return np.concatenate([pt, np.full((n, pt.shape[1]), -1, np.int32)]), np.concatenate([ptr, np.full(n, ptr[-1], np.int32)])


@pytest.mark.parametrize("kind,d,hq,hkv,ctx,rows,max_rows,window,sinks", [c for c in WINDOW_CASES if c[6] >= 130])
def test_window_prefill_matches_the_definition(kind, d, hq, hkv, ctx, rows, max_rows, window, sinks):
    say(f"attn_window kv8 prefill {kind} d={d} hq={hq} hkv={hkv} ctx={ctx} rows={rows} window={window} sinks={sinks}")
    pt, ptr, pos, pages = _batch(ctx, rows, d + hq, extra_rows=2)
    pt, ptr = _with_empty_requests(pt, ptr, max_rows, hq, hkv, window, sinks)
    _check_window(kind, d, hq, hkv, pt, ptr, pos, pages, max_rows, window, sinks, 3 * d + hq)


@pytest.mark.parametrize("kind,d,hq,hkv,ctx,rows", [("bf16", 128, 4, 1, [333, 64], [200, 64]), ("f16", 128, 7, 1, [700], [150]),
                                                    ("bf16", 64, 16, 2, [400, 33], [260, 33]), ("bf16", 256, 4, 2, [900, 1], [50, 1])])
@pytest.mark.parametrize("window,sinks", [(2**31 - 1, 0), (0, 1 << 30), (1 << 24, 3)])
def test_window_split_pages(kind, d, hq, hkv, ctx, rows, window, sinks):
    say(f"attn_window kv8 split {kind} d={d} hq={hq} hkv={hkv} ctx={ctx} rows={rows} window={window} sinks={sinks}")
    pt, ptr, pos, pages = _batch(ctx, rows, d + hq, extra_rows=2, stride_extra=30000)
    _check_window(kind, d, hq, hkv, pt, ptr, pos, pages, max(rows), window, sinks, 3 * d + hq)


@pytest.mark.parametrize("max_rows", [5, 200])
@pytest.mark.parametrize("prefill", [False, True])
def test_window_odd_rows(max_rows, prefill):
    """Unsorted and repeated positions, padding rows, positions past the page table, pages that are none, rows past max_rows."""
    say(f"attn_window kv8 odd rows max_rows={max_rows} prefill={prefill}")
    pt, ptr, pos, pages = _batch([400, 300, 260], [7, 203, 4], 5, extra_rows=1, stride_extra=0)
    rng = np.random.default_rng(2)
    pos[:7] = [399, -1, 20, 20, 150, 5000, 0]
    pos[7:210] = rng.integers(-3, 300, 203)
    pt[0, 1], pt[1, 2], pt[2, 0] = -1, pages, 2 ** 30
    if prefill:
        pt, ptr = _with_empty_requests(pt, ptr, max_rows, 8, 2, 90, 70)
    _check_window("bf16", 128, 8, 2, pt, ptr, pos, pages, max_rows, 90, 70, 17)


@pytest.mark.parametrize("rows,prefill", [(5, False), (150, False), (150, True)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_window_masked_nan(rows, prefill, d):
    """Slots of positions that some rows of a tile see and others do not hold NaN: only the rows that see them show it."""
    say(f"attn_window kv8 masked NaN rows={rows} prefill={prefill} d={d}")
    pt, ptr, pos, pages = _batch([200], [rows], 8)
    at = np.array([pt[0, p // 64] * 64 + p % 64 for p in (198, 199, 90)])
    if prefill:
        pt, ptr = _with_empty_requests(pt, ptr, rows, 4, 1, 60, 4)
    _check_window("bf16", d, 4, 1, pt, ptr, pos, pages, rows, 60, 4, 23, poison=at)


@pytest.mark.parametrize("rows,prefill", [(5, False), (150, False), (150, True)])
def test_values_past_fp16(rows, prefill):
    """In fp16 a large scale makes infinities of large codes, in V: they reach the rows that see them and no others."""
    say(f"attn_window kv8 past fp16 rows={rows} prefill={prefill}")
    pt, ptr, pos, pages = _batch([200], [rows], 8)
    exps = np.full((pages, 1, 2), -5)
    exps[pt[0, 3], 0, 1] = 9                                     # positions 192 .. 199
    if prefill:
        pt, ptr = _with_empty_requests(pt, ptr, rows, 4, 1, 60, 4)
    cache, K, V = _cache(pages, 1, 128, 4, exps=exps)
    V = torch.from_numpy(V).to(torch.float16).double().numpy()   # as the queries' type holds them
    assert np.isinf(V).any()
    q, out, lse = _queries(rows, 4, 128, "f16", 2)
    res, n = _window_want(_f64(q), K, V, pt, ptr, pos, pages, rows, 60, 4, 0.09)
    bst.attn_window(q, cache, *[torch.from_numpy(x).cuda() for x in (pt, ptr, pos)], rows, 60, 4, out[:rows, :4], scale=0.09,
                    lse=lse[:rows], workspace=bst.attn_workspace("cuda"))
    check_rows(_f64(out[:rows, :4]), _f64(lse[:rows]), res, "f16", n, np.max(np.abs(V[np.isfinite(V)])))


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
@pytest.mark.parametrize("rows", [2, 40])
def test_any_finite_scale(scale, rows):
    pt, ptr, pos, pages = _batch([200], [rows], 4)
    cache, K, V = _cache(pages, 2, 128, 12)
    q, out, lse = _queries(rows, 8, 128, "bf16", 3)
    res, n = _window_want(_f64(q), K, V, pt, ptr, pos, pages, rows, 70, 3, scale)
    bst.attn_window(q, cache, *[torch.from_numpy(x).cuda() for x in (pt, ptr, pos)], rows, 70, 3, out[:rows, :8], scale=scale,
                    lse=lse[:rows], workspace=bst.attn_workspace("cuda"))
    check_rows(_f64(out[:rows, :8]), _f64(lse[:rows]), res, "bf16", n, np.abs(V).max())


def test_pools_past_4_gib():
    say("kv8 pool past 4 GiB")
    hkv, d = 8, 128
    pages = ((1 << 32) // (hkv * 2 * d)) // 64 + 1000
    cache = bst.KV8Cache.empty(pages, hkv, d, "cuda")
    far = np.concatenate([(pages - 1) * 64 + np.arange(64), np.arange(40), (pages - 2) * 64 + np.arange(64)])
    k, v = (torch.randn((168, hkv, d), generator=_gen(i), device="cuda").bfloat16() for i in (1, 2))
    bst.kv8_store(k, v, _i32(far), cache)
    ref = Kv8(3, hkv, d)
    near = np.concatenate([np.arange(64), 64 + np.arange(40), 128 + np.arange(64)])
    ref.store(_f64(k), _f64(v), near)
    K, V = (x[near] for x in ref.values())
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    bst.kv8_load(cache, _i32(far), ko, vo)
    np.testing.assert_array_equal(_f64(ko), K), np.testing.assert_array_equal(_f64(vo), V)
    q, out, lse = _queries(1, 16, d, "bf16", 4)
    bst.attn_slots(q, cache, _i32(far).view(1, -1), out[:1, :16], lse=lse[:1])
    check_rows(_f64(out[:1, :16]), _f64(lse[:1]), [attend_row(_f64(q[0]), K, V, d ** -0.5)], "bf16", [168], np.abs(V).max())
    page = _i32([[pages - 1, pages - 2, 0]])                     # the same as positions of a request
    order = np.concatenate([np.arange(64), 104 + np.arange(64), 64 + np.arange(22)])
    for rows, req in ((1, 1), (150, 1), (150, 4000)):
        q, out, lse = _queries(rows, 16, d, "bf16", 4)
        pos, ptr = torch.arange(150 - rows, 150, dtype=torch.int32, device="cuda"), _i32([0] + [rows] * req)
        bst.attn_window(q, cache, page.expand(req, 3).contiguous(), ptr, pos, rows, 1000, 0, out[:rows, :16], lse=lse[:rows],
                        workspace=bst.attn_workspace("cuda"))
        some = [0, rows // 2, rows - 1]
        want = [attend_row(_f64(q[r]), K[order[:int(pos[r]) + 1]], V[order[:int(pos[r]) + 1]], d ** -0.5) for r in some]
        check_rows(_f64(out[some, :16]), _f64(lse[some]), want, "bf16", [150] * 3, np.abs(V).max())
    del cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("case", ["slots", "window_decode", "window_prefill", "store"])
def test_captured_calls_replay_like_eager(case):
    say(f"kv8 graph {case}")
    hkv, hq, d = 2, 16, 128
    pt, ptr, pos, pages = _batch([700, 260], [1, 1] if case != "window_prefill" else [300, 200], 3)
    rows = len(pos)
    cache, _, _ = _cache(pages, hkv, d, 5)
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
            bst.kv8_store(kin, kin, at, cache)
            bst.kv8_load(cache, at, ko, vo)
        else:
            bst.attn_window(q, cache, *meta, 1 if case == "window_decode" else 300, 150, 4, out, lse=lse, workspace=ws)

    kept = cache.codes.clone(), cache.scales.clone()

    def fill(i):
        q.copy_(torch.randn(q.shape, generator=_gen(50 + i), device="cuda"))
        kin.copy_(torch.randn(kin.shape, generator=_gen(90 + i), device="cuda") * 2.0 ** i)
        cache.codes.copy_(kept[0]), cache.scales.copy_(kept[1])

    result = lambda: [x.clone() for x in ((ko, vo, cache.codes, cache.scales) if case == "store" else (out, lse))]  # noqa: E731
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


def test_prepared_calls():
    cache, _, _ = _cache(4, 2, 128, 5)
    k, v = _rows(50, 2, 128, "bf16", 6, True)
    slots = _i32(np.arange(64, 114))
    for call in (bst.prepare_kv8_store(k, v, slots, cache), bst.prepare_kv8_store(k, v, slots, cache).bind()):
        cache.codes.zero_(), cache.scales.fill_(2.0 ** -120)
        call()
        got = cache.codes.clone()
        cache.codes.zero_(), cache.scales.fill_(2.0 ** -120)
        bst.kv8_store(k, v, slots, cache)
        assert torch.equal(got, cache.codes)
    a, b = (torch.empty((50, 2, 128), dtype=torch.float32, device="cuda") for _ in range(2))
    bst.prepare_kv8_load(cache, slots, a, b)()
    c, d = torch.empty_like(a), torch.empty_like(b)
    bst.kv8_load(cache, slots, c, d)
    assert torch.equal(a, c) and torch.equal(b, d)
