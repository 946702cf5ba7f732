"""The 4-bit index keys on the GPU: stored codes and compressed keys exact, scores
within the bound that more_ref.py derives, and a run of everything as a serving
loop uses it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scoring_top_amd as bst
import synth
from attn_ref import attend_row, check_rows, dequantise, quantise
from block_scoring_top_amd.pipeline import IndexerPath, PagedBatch
from gpu_util import say
from more_ref import Kv8, compressed_keys, score_row
from synth.device import upload, upload_compress

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


@pytest.mark.parametrize("T,kind,c,wide", [(1, "bf16", 1, False), (3, "f32", 4, True), (64, "bf16", 1, True), (257, "f16", 4, False),
                                           (1003, "f32", 1, False), (5000, "bf16", 4, True)])
def test_store_and_load_match_the_definition(T, kind, c, wide):
    say(f"idx4 T={T} {kind} c={c} wide={wide}")
    rng = np.random.default_rng(T)
    pages = T // (64 // c) + 2
    n = pages * (64 // c)
    x = torch.tensor(rng.standard_normal((T, 160 if wide else 128)) * np.exp(2 * rng.standard_normal((T, 1)))).to(TYPES[kind]).cuda()
    x = x[:, 16:144] if wide else x
    slots = rng.permutation(n)[:T]
    if T > 10:
        slots[::7], slots[T // 2] = -1, n
    cache = bst.Idx4Cache(torch.full((n, 64), 0xA5, dtype=torch.uint8, device="cuda"),
                          torch.full((n, 4), 0x5A, dtype=torch.uint8, device="cuda"), c)
    bst.idx4_store(x, _i32(slots), cache)
    torch.cuda.synchronize()
    want_c, want_s = np.full((n, 64), 0xA5, np.uint8), np.full((n, 4), 0x5A, np.uint8)
    ok = (slots >= 0) & (slots < n)
    cc, ss = quantise(_f64(x))
    want_c[slots[ok]], want_s[slots[ok]] = cc[ok], ss[ok]
    np.testing.assert_array_equal(cache.codes.cpu().numpy(), want_c)
    np.testing.assert_array_equal(cache.scales.cpu().numpy(), want_s)
    rd = np.concatenate([slots[rng.permutation(T)], slots[:1], [-1, n]])
    for out_kind in TYPES:
        out = torch.full((len(rd), 136), 7.0, dtype=TYPES[out_kind], device="cuda")
        bst.idx4_load(cache, _i32(rd), out[:, :128])
        ok = (rd >= 0) & (rd < n)
        want = np.zeros((len(rd), 128))
        want[ok] = dequantise(want_c[rd[ok]], want_s[rd[ok]])
        np.testing.assert_array_equal(_f64(out[:, :128]), _f64(torch.from_numpy(want).to(TYPES[out_kind])))
        assert (out[:, 128:] == 7.0).all()


def test_store_special_values():
    rows = np.zeros((8, 128))
    rows[1], rows[2, :32], rows[2, 32:64], rows[3, 5], rows[4, 40], rows[5, 70] = 3e38, 2.0 ** -130, 2.0 ** -126, np.inf, -np.inf, np.nan
    rows[6] = np.tile([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 7.9, -0.25, -5.0, 0.0, -0.0, 6.5, 1.0], 8)
    rows[7] = rows[6] * 2.0 ** -20
    x = torch.tensor(rows, dtype=torch.float32, device="cuda")
    cache = bst.Idx4Cache.empty(1, 4, "cuda")
    bst.idx4_store(x, _i32(np.arange(8)), cache)
    c, s = quantise(_f64(x))
    np.testing.assert_array_equal(cache.codes[:8].cpu().numpy(), c)
    np.testing.assert_array_equal(cache.scales[:8].cpu().numpy(), s)
    e = torch.empty((0, 128), device="cuda")
    bst.idx4_store(e, _i32([]), cache)
    bst.idx4_load(cache, _i32([]), e)


def _compress_want(ci, k_raw, ring, ring_pos):
    """{key slot: key in bf16} of the blocks that the call completes."""
    raws, poss, at = [], [], []
    for b in range(len(ci.tok_start)):
        t0, n, start = int(ci.req_tok_ptr[b]), int(ci.req_tok_ptr[b + 1] - ci.req_tok_ptr[b]), int(ci.tok_start[b])
        for j in range(start // 4, (start + n) // 4):
            raws.append([k_raw[t0 + 4 * j + u - start] if 4 * j + u >= start else ring[b, u] for u in range(4)])
            first = 4 * j - start
            poss.append([4 * j] * 3 if ci.mrope_pos is None else ci.mrope_pos[t0 + first] if first >= 0 else ring_pos[b])
            at.append(int(ci.page_table[b][4 * j // 64]) * 16 + j % 16)
    return np.array(at), compressed_keys(np.array(raws), np.array(poss), ci.rotary_dim, ci.sections, ci.theta)


@pytest.mark.parametrize("make", [lambda: synth.qsa_compress_decode_64req(), lambda: synth.qsa_compress_prefill_8k()])
def test_compress_store_matches_the_definition(make):
    """Codes and scales of every completed block; rings and their positions as idx_compress_store leaves them; nothing else
    touched.  The reference's and the kernel's values lie within 2^-29 of each other before they are rounded: none of these
    fixed inputs has an element so near to a tie."""
    ci = make()
    say(f"idx4 compress {getattr(ci, 'name', '?')} tokens={ci.num_tok}")
    a, b = upload_compress(ci, "cuda"), upload_compress(ci, "cuda")
    values = lambda t: _f64(t.view(torch.bfloat16))  # noqa: E731
    at, keys = _compress_want(ci, values(b.k_raw), values(b.ring), b.ring_pos.cpu().numpy())
    bst.idx_compress_store(*a.args())
    n = a.kcache.shape[0]
    cache = bst.Idx4Cache(torch.full((n, 64), 0xA5, dtype=torch.uint8, device="cuda"),
                          torch.full((n, 4), 0x5A, dtype=torch.uint8, device="cuda"), 4)
    bst.idx4_compress_store(*list(b.args())[:-2], cache)
    torch.cuda.synchronize()
    assert torch.equal(a.ring, b.ring) and torch.equal(a.ring_pos, b.ring_pos)
    codes, scales = np.full((n, 64), 0xA5, np.uint8), np.full((n, 4), 0x5A, np.uint8)
    codes[at], scales[at] = quantise(keys)
    np.testing.assert_array_equal(cache.codes.cpu().numpy(), codes)
    np.testing.assert_array_equal(cache.scales.cpu().numpy(), scales)


def test_compress_store_special_values():
    """Blocks of zeros, of one nonzero channel, near the ends of the range, and with infinities and NaN: zeros stay
    zeros, and a key that is not finite is NaN throughout."""
    raw = torch.zeros((32, 128))
    raw[4:8, 5] = 3.0
    raw[8:12] = 3e38 * torch.linspace(-1, 1, 128)
    raw[12:16] = 1e-38 * torch.linspace(-1, 1, 128)
    raw[16, 7], raw[21, 100], raw[24:28] = float("inf"), float("nan"), 1.5
    raw[28:32] = torch.randn((4, 128), generator=torch.Generator().manual_seed(1))
    raw = raw.bfloat16()
    cache = bst.Idx4Cache.empty(1, 4, "cuda")
    ring = torch.zeros((1, 4, 128), dtype=torch.int16, device="cuda")
    bst.idx4_compress_store(raw.view(torch.int16).cuda(), _i32([0, 32]), _i32([0]), None, 32, 128, (64, 0, 0), 10000.0, ring, None,
                            _i32([[0]]), cache)
    scales = cache.scales.cpu().numpy()
    assert (scales[4:6] == 255).all()
    ok = [0, 1, 3, 6, 7]                                         # the sum of block 2 leaves FP32
    keys = compressed_keys(_f64(raw).reshape(8, 4, 128)[ok], np.repeat(4 * np.array(ok)[:, None], 3, 1), 128, (64, 0, 0), 10000.0)
    c, s = quantise(keys)
    np.testing.assert_array_equal(cache.codes.cpu().numpy()[ok], c)
    np.testing.assert_array_equal(scales[ok], s)
    assert (scales[2] == 255).all()


def _score_case(c, ctx, rows, seed, spread=0.0, max_vis=None, extra=0):
    rng = np.random.default_rng(seed)
    pages = [max(1, -(-t // 64)) for t in ctx]
    perm = rng.permutation(sum(pages))
    pt = np.full((len(ctx), max(pages) + 1), -1, np.int32)
    at = 0
    for b, p in enumerate(pages):
        pt[b, :p] = perm[at:at + p]
        at += p
    ptr = np.concatenate([[0], np.cumsum(rows)])
    pos = np.concatenate([np.arange(t - n, t) for t, n in zip(ctx, rows)] + [np.full(extra, 3)])
    n = sum(pages) * (64 // c)
    k = rng.standard_normal((n, 128)) * np.exp(spread * rng.standard_normal((n, 4, 1)).repeat(32, 2).reshape(n, 128))
    kc, ks = quantise(k)
    q = torch.tensor(rng.standard_normal((len(pos), 4, 128)) * np.exp(spread * rng.standard_normal((len(pos), 4, 1)))).bfloat16()
    return pt, ptr, pos, kc, ks, q, (max(ctx) // c if max_vis is None else max_vis)


def _check_scores(c, pt, ptr, pos, kc, ks, q, max_vis, ld=None, lost=()):
    """Scores, lengths, and every entry that is not to be written; lost: (request, logical page) without a page."""
    cache = bst.Idx4Cache(torch.from_numpy(kc).cuda(), torch.from_numpy(ks).cuda(), c)
    rows, ld = len(pos), ld or max(1, max_vis)
    scores = torch.full((rows + 1, ld), -77.0, dtype=torch.float32, device="cuda")
    row_len = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    bst.idx4_score(q.cuda(), cache, _i32(pt), _i32(ptr), _i32(pos), max_vis, scores[:rows], row_len)
    torch.cuda.synchronize()
    got, n_got = scores.cpu().numpy(), row_len.cpu().numpy()
    K = dequantise(kc, ks)
    Q = dequantise(*quantise(_f64(q)))
    want = np.full((rows + 1, ld), -77.0)
    bound = np.zeros((rows + 1, ld))
    for b in range(len(ptr) - 1):
        for r in range(ptr[b], ptr[b + 1]):
            n = max(0, min((int(pos[r]) + 1) // c, max_vis))
            assert n_got[r] == n
            j = np.arange(n)
            page = pt[b][j * c // 64]
            at = np.where((page >= 0) & (page < kc.shape[0] // (64 // c)), page, 0).astype(np.int64) * (64 // c) + j % (64 // c)
            if n:
                want[r, :n], bound[r, :n] = score_row(np.nan_to_num(Q[r]), np.nan_to_num(K[at]))
            for req, lp in lost:                                 # unspecified
                if req == b:
                    u = j[j * c // 64 == lp]
                    want[r, u] = got[r, u]
    err = np.abs(got - want)
    assert (err <= bound).all(), f"{(err > bound).sum()} off, worst {np.nanmax(err - bound)}"


SCORE_CASES = [  # c, contexts, rows
    (1, [1], [1]), (4, [3], [1]), (4, [4], [1]), (1, [64, 65, 130], [1, 1, 1]), (4, [8194], [1]), (4, [700, 64, 3, 260], [4, 1, 3, 2]),
    (1, [500, 70], [4, 3]), (4, [1500, 40, 900], [6, 5, 6]), (1, [333, 90], [8, 6]), (4, [2000, 300], [9, 9]),
    (1, [600], [17]), (4, [3000], [130]), (1, [700, 200, 20], [129, 64, 1]), (4, [9000, 500], [300, 33]), (1, [1100], [1000]),
    (4, [400] * 20, [0, 1] * 10), (4, [900] * 70, [1] * 63 + [700, 0, 40] + [1] * 4), (1, [300] * 130, [40] * 130),
    (1, [2100, 90], [30, 2]), (4, [1300] * 9, [0, 0, 33, 0, 64, 1, 31, 32, 90]), (1, [5000] * 64, [1] * 64), (4, [70000] * 16, [2] * 16), (4, [33000] * 32, [6] * 32)]


@pytest.mark.parametrize("c,ctx,rows", SCORE_CASES)
@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_scores_match_the_definition(c, ctx, rows, spread):
    say(f"idx4_score c={c} contexts={ctx[:4]} rows={rows[:4]} requests={len(ctx)} spread={spread}")
    case = _score_case(c, ctx, rows, sum(ctx) + sum(rows), spread)
    _check_scores(c, *case)


@pytest.mark.parametrize("c,ctx,rows", [(4, [9000, 700] * 35, [1, 0] * 34 + [600, 1]), (1, [300, 1200, 100, 1300], [1, 64, 0, 1] * 1),
                                        (1, [900] * 40 + [400] * 30, [65] + [1] * 38 + [200] + [0, 1] * 15),
                                        (4, [2000] * 130, [1] * 64 + [129] + [3] * 65), (1, [500] * 7, [0, 0, 130, 0, 0, 0, 0])])
def test_scores_of_long_requests_among_short_ones(c, ctx, rows):
    """At most 20 rows a request on average: the kernel for few rows, in which blocks past a request's first 64 rows are
    others' work."""
    assert sum(rows) <= 20 * len(rows)
    say(f"idx4 c={c} {len(ctx)} requests rows={max(rows)}")
    _check_scores(c, *_score_case(c, ctx, rows, sum(rows)))


@pytest.mark.parametrize("c,ctx,rows", [(1, [4000, 70, 2500], [1500, 40, 1200]), (4, [12001, 900, 5], [3000, 500, 2]), (1, [10241], [700]),
                                        (4, [33000, 16500, 4100], [20, 700, 1100]), (1, [257, 1025, 30] * 20, [200, 130, 7] * 20)])
def test_scores_of_many_rows(c, ctx, rows):
    """Large grids: workgroups of several stages, the last of them cut by the context, by the rows or by causality."""
    say(f"idx4 c={c} {ctx[:3]} rows={rows[:3]}")
    _check_scores(c, *_score_case(c, ctx, rows, sum(rows)))


@pytest.mark.parametrize("rows", [[1, 2], [6, 8], [100, 40]])
@pytest.mark.parametrize("c", [1, 4])
def test_scores_odd_rows(rows, c):
    """Positions in any order, before the first block and past max_vis; rows behind the last request; odd strides (no
    16-byte stores); pages that hold nothing."""
    say(f"idx4_score odd rows={rows} c={c}")
    for max_vis, ld in ((201, 201), (7, 13), (130, 131), (0, 5)):
        pt, ptr, pos, kc, ks, q, _ = _score_case(c, [1000, 650], rows, c + max_vis, extra=2)
        rng = np.random.default_rng(5)
        pos[:-2] = rng.integers(-5, 1000, len(pos) - 2)
        pt[0, 1], pt[1, 0], pt[1, 9] = -1, 2 ** 30, 99
        _check_scores(c, pt, ptr, pos, kc, ks, q, max_vis, ld, lost=((0, 1), (1, 0), (1, 9)))


def test_groups_of_nan_count_as_nothing():
    say("idx4_score NaN groups")
    for rows in ([2], [40]):
        pt, ptr, pos, kc, ks, q, vis = _score_case(1, [300], rows, 4)
        ks[5, 2], kc[5, 32:48] = 255, 0
        ks[70] = 255
        q[0, 1, 40], q[1, 3, 0], q[1, 2, 127] = float("nan"), float("inf"), -float("inf")
        cache = bst.Idx4Cache(torch.from_numpy(kc).cuda(), torch.from_numpy(ks).cuda(), 1)
        scores = torch.full((len(pos), vis), -77.0, device="cuda")
        bst.idx4_score(q.cuda(), cache, _i32(pt), _i32(ptr), _i32(pos), vis, scores)
        got = scores.cpu().numpy()
        K, Q = dequantise(kc, ks), dequantise(*quantise(_f64(q)))
        for r in range(len(pos)):
            n = int(pos[r]) + 1
            at = pt[0][np.arange(n) // 64].astype(np.int64) * 64 + np.arange(n) % 64
            x = Q[r] @ K[at].T
            want = np.where(np.isnan(x), 0.0, np.maximum(x, 0.0)).sum(0) / np.sqrt(128.0)
            bound = 136 * 2.0 ** -24 * (np.abs(np.nan_to_num(Q[r])) @ np.abs(np.nan_to_num(K[at])).T).sum(0) / np.sqrt(128.0)
            assert (np.abs(got[r, :n] - want) <= bound).all(), r


@pytest.mark.parametrize("rows", [3, 70])
def test_scales_over_their_whole_range(rows):
    """Keys and queries of 2^-118 to 2^120, whose products leave FP32's range on both sides.  Beside the bound, what may be
    lost below its least normal number: 2^-126 for each of 4 x 128 products and as many sums, over sqrt(128)."""
    say(f"idx4 scales rows={rows}")
    rng = np.random.default_rng(rows)
    pt, ptr, pos, kc, ks, q, vis = _score_case(1, [700], [rows], 2)
    K = dequantise(kc, ks) * np.ldexp(1.0, rng.integers(-118, 118, (len(kc), 1)))
    kc, ks = quantise(K)
    q = (q.double() * torch.tensor(np.ldexp(1.0, rng.integers(-118, 118, (rows, 1, 1))))).bfloat16()
    cache = bst.Idx4Cache(torch.from_numpy(kc).cuda(), torch.from_numpy(ks).cuda(), 1)
    scores = torch.full((rows, vis), -77.0, device="cuda")
    bst.idx4_score(q.cuda(), cache, _i32(pt), _i32(ptr), _i32(pos), vis, scores)
    got = scores.cpu().numpy().astype(np.float64)
    K, Q, finite = dequantise(kc, ks), dequantise(*quantise(_f64(q))), 0
    for r in range(rows):
        j = np.arange(pos[r] + 1)
        k = K[pt[0][j // 64].astype(np.int64) * 64 + j % 64]
        want, bound = score_row(Q[r], k)
        mag = (np.abs(Q[r]) @ np.abs(k).T).sum(0)
        small = mag < 2.0 ** 127                                 # no sum on the way leaves the range
        finite += small.sum()
        err = np.abs(np.where(small, got[r, j] - want, 0.0))
        assert (err <= bound + 4 * 256 * 2.0 ** -126 / np.sqrt(128.0)).all(), (r, err.max())
        assert not np.isnan(got[r, j]).any() and (got[r, j] >= 0).all()
    assert finite > 300


def test_caches_past_4_gib():
    """Keys whose byte offsets pass 32 bits."""
    say("idx4 past 4 GiB")
    pages = (1 << 32) // (64 * 64) + 1000                        # c = 1
    cache = bst.Idx4Cache.empty(pages, 1, "cuda")
    rng = np.random.default_rng(1)
    k = torch.tensor(rng.standard_normal((192, 128)), dtype=torch.float32, device="cuda")
    pt = np.array([[pages - 1, 0, pages - 7]], np.int32)
    slots = (pt[0][:, None].astype(np.int64) * 64 + np.arange(64)).ravel()
    bst.idx4_store(k, _i32(slots), cache)
    out = torch.empty_like(k)
    bst.idx4_load(cache, _i32(slots), out)
    K = dequantise(*quantise(_f64(k)))
    np.testing.assert_array_equal(_f64(out), K)
    for rows in (1, 6, 150):
        q = torch.tensor(rng.standard_normal((rows, 4, 128))).bfloat16()
        scores = torch.zeros((rows, 192), device="cuda")
        bst.idx4_score(q.cuda(), cache, _i32(pt), _i32([0, rows]), _i32([191] * rows), 192, scores)
        for r in (0, rows - 1):
            want, bound = score_row(dequantise(*quantise(_f64(q[r]))), K)
            assert (np.abs(_f64(scores[r]) - want) <= bound).all()
    del cache
    torch.cuda.empty_cache()


def test_captured_scores_replay_like_eager():
    for rows in ([1, 1], [6, 6], [300, 20]):
        pt, ptr, pos, kc, ks, q, vis = _score_case(4, [3000, 1700], rows, 9)
        cache = bst.Idx4Cache(torch.from_numpy(kc).cuda(), torch.from_numpy(ks).cuda(), 4)
        x, scores = torch.empty_like(q, device="cuda"), torch.zeros((len(pos), vis), device="cuda")
        keep = [_i32(v) for v in (pt, ptr, pos)]
        call = bst.prepare_idx4_score(x, cache, *keep, vis, scores)
        qs = [q, -q, q.flip(0)]
        want = []
        for y in qs:
            x.copy_(y)
            call()
            torch.cuda.synchronize()
            want.append(scores.clone())
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        torch.cuda.synchronize()
        for rep in range(2):
            for y, w in zip(qs, want):
                x.copy_(y)
                scores.fill_(0)
                torch.cuda.synchronize()
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(scores, w)


def test_path_scores_and_selects_over_4_bits():
    """IndexerPath with the "idx4" scorer: its selection is the exact top-k of the scores that it wrote."""
    inp = synth.qsa_verify_64req(B=4, lo=300, hi=9000)
    dev = upload(inp, "cuda")
    n = dev.kcache.shape[0] if dev.kcache.dim() == 2 else dev.kcache.numel() // 128
    cache = bst.Idx4Cache.empty(inp.num_pages, inp.c, "cuda")
    bst.idx4_store(dev.kcache.view(torch.bfloat16).view(-1, 128)[:cache.num_keys], _i32(np.arange(cache.num_keys)), cache)
    assert n >= cache.num_keys
    dev.kcache = cache
    p = IndexerPath(dev, "idx4")
    p.run()
    torch.cuda.synchronize()
    first = p.slots.clone()
    for r in range(inp.num_rows):
        m = int(p.row_len[r])
        take = min(m, inp.k)
        s = p.scores[r, :m]
        order = torch.argsort(s, descending=True, stable=True)[:take]
        assert set(p.sel[r, :take].tolist()) == set(order.tolist())
    p.run(fused=False)
    torch.cuda.synchronize()
    assert torch.equal(first.sort(1).values, p.slots.sort(1).values)
    with pytest.raises(ValueError):
        IndexerPath(type("X", (), dict(vars(dev), kcache=bst.Idx4Cache.empty(4, 1, "cuda"), c=4, q=dev.q))(), "idx4")


def test_a_serving_loop_of_the_new_calls():
    """Prompts and decode steps of four requests (c = 1): pages, K/V in 8 bits, index keys in 4, scores, selection and
    attention, one request finished and another begun in its pages; every step's attention against 64 bits over the
    reference caches, at the slots that the selection chose."""
    say("serving loop")
    B, hkv, hq, d, k, cap = 4, 2, 8, 128, 64, 700
    rng = np.random.default_rng(7)
    batch = PagedBatch(B, cap, 30, 800, "cuda")
    cache, keys = bst.KV8Cache.empty(30, hkv, d, "cuda"), bst.Idx4Cache.empty(30, 1, "cuda")
    ref = Kv8(30, hkv, d)
    steps = [[300, 70, 0, 129], [1, 1, 200, 1], [1, 6, 1, 1], [1, 1, 1, 1], [64, 1, 0, 1]]
    finish = {2: [-1, 0, -1, 130]}
    for i, new in enumerate(steps):
        batch.extend(_i32(new))
        ptr = batch.req_row_ptr.cpu().numpy()
        rows = int(ptr[-1])
        kk, vv = (torch.tensor(rng.standard_normal((rows, hkv, d)) * (i + 1)).bfloat16().cuda() for _ in range(2))
        ik = torch.tensor(rng.standard_normal((rows, 128))).bfloat16().cuda()
        slots = batch.slots[:rows]
        bst.kv8_store(kk, vv, slots, cache)
        bst.idx4_store(ik, slots, keys)
        ref.store(_f64(kk), _f64(vv), slots.cpu().numpy())
        inp = type("Inputs", (), dict(c=1, k=k, q=torch.tensor(rng.standard_normal((rows, 4, 128))).bfloat16().cuda(), kcache=keys,
                                      num_pages=30, page_table=batch.page_table, req_row_ptr=batch.req_row_ptr,
                                      row_pos=batch.row_pos[:rows], max_vis=cap))()
        p = IndexerPath(inp, "idx4")
        p.run()
        q = torch.tensor(rng.standard_normal((rows, hq, d))).bfloat16().cuda()
        out, lse = torch.empty_like(q), torch.empty((rows, hq), dtype=torch.float32, device="cuda")
        p.attend(q, cache, out, lse=lse)
        torch.cuda.synchronize()
        K, V = ref.values()
        table, pos = batch.page_table.cpu().numpy(), batch.row_pos.cpu().numpy()
        chosen, cnt = p.slots.cpu().numpy(), p.out_count.cpu().numpy()
        want, n = [], []
        for r in range(rows):
            b = int(np.searchsorted(ptr, r, side="right") - 1)
            s = chosen[r, :cnt[r]]
            assert len(s) == min(k, pos[r] + 1) and len(set(s)) == len(s)
            seen = {int(table[b, t // 64]) * 64 + t % 64 for t in range(pos[r] + 1)}
            assert set(s.tolist()) <= seen
            want.append(attend_row(_f64(q[r]), K[s], V[s], d ** -0.5))
            n.append(len(s))
        check_rows(_f64(out), _f64(lse), want, "bf16", n, np.abs(V).max())
        if i in finish:
            batch.release(_i32(finish[i]))
    assert batch.kv_len.tolist()[0] == 367 and batch.pool.state.tolist()[2] == 0
