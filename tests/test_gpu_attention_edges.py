"""The attention calls at the edges of their types and sizes, against the 64-bit
references of attn_ref.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scoring_top_amd as bst
from attn_ref import attend_row, check_rows, dequantise, quantise
from gpu_util import say
from test_gpu_attention import TYPES, _batch, _cache, _f64, _gen, _queries, _window_want

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- infinities in split keys

def _infinite_values(cache, V, slots):
    """Puts infinities of both signs into V at `slots` (never into K); V receives what the kernels see.  The 4-bit cache
    holds none, but a large scale leaves fp16's range."""
    if isinstance(cache, bst.KV16Cache):
        for s, x in zip(slots, (np.inf, -np.inf) * len(slots)):
            cache.v[s, :, 3::7] = x
            V[s, :, 3::7] = x
        return V
    at = torch.as_tensor(slots, device="cuda")
    cache.scales[at, :, 1] = 127 + 15                            # 2^15: codes from 2 on stand for 65,536 and more
    c = cache.codes[at, :, 1].cpu().numpy()
    c = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
    v = np.where(c >= 8, -1.0, 1.0) * np.array([0, .5, 1, 1.5, 2, 3, 4, 6])[c & 7] * 2.0 ** 15
    V[slots] = np.where(np.abs(v) > 65504, np.copysign(np.inf, v), v)
    return V


# Parts of a row's keys by the splitting rule: (rows, entries) -> 2, 4, 8, 16 parts, for each column layout that joins
# in its own way (a tile of up to 8, of 16 and of 28 columns, head_dim 64, 128 and 256).
@pytest.mark.parametrize("kind,form,d,hq,hkv,rows,n", [
    ("bf16", "kv16", 128, 16, 2, 64, 2051), ("bf16", "kv16", 128, 16, 1, 100, 2051), ("bf16", "kv16", 128, 16, 1, 64, 2051),
    ("f16", "kv16", 128, 28, 1, 100, 2051), ("f16", "kv16", 128, 28, 1, 150, 2051), ("bf16", "kv16", 128, 4, 1, 100, 600),
    ("bf16", "kv16", 256, 16, 1, 8, 200), ("bf16", "kv16", 256, 28, 1, 33, 600), ("f16", "kv16", 64, 16, 1, 33, 2051),
    ("f16", "kv16", 64, 28, 1, 64, 2051), ("bf16", "kv16", 128, 16, 2, 16, 2051), ("bf16", "kv16", 128, 16, 2, 1, 2051),
    ("f16", "kv4", 128, 16, 2, 100, 2051), ("f16", "kv4", 128, 16, 1, 64, 2051), ("f16", "kv4", 64, 28, 1, 150, 2051)])
@pytest.mark.parametrize("window", [False, True])
def test_split_keys_pass_an_infinity_on(kind, form, d, hq, hkv, rows, n, window):
    """An infinity in V that a row sees is its result, wherever in the row's keys it lies and however many parts they
    are split into: in the last part (joined with copies of itself of weight 0), the first, and one between."""
    say(f"infinite values in split keys {kind} {form} d={d} hq={hq} hkv={hkv} rows={rows} n={n} window={window}")
    scale = 0.09
    if window and (hq // hkv > 16 or rows > 64):
        rows = min(rows, 64)                                     # decode rows, one request each
    pages = -(-n // 64) + 3
    cache, K, V = _cache(form, kind, pages, hkv, d, 7)
    q, out, lse = _queries(rows, hq, d, kind, 5)
    rng = np.random.default_rng(n)
    if window:                                                   # every request reads the same pages
        pt = np.tile(rng.permutation(pages)[:-(-n // 64)].astype(np.int32), (rows, 1))
        ptr, pos = np.arange(rows + 1, dtype=np.int32), np.full(rows, n - 1, np.int32)
        lists = np.tile(pt[0][np.arange(n) // 64] * 64 + np.arange(n) % 64, (rows, 1))
    else:
        lists = np.stack([rng.permutation(pages * 64)[:n] for _ in range(rows)]).astype(np.int32)
        lists[:, [0, n // 3, n - 1]] = lists[0, [0, n // 3, n - 1]]
    for where in (n - 1, 0, n // 3):
        if form == "kv16":
            pool = torch.stack([cache.k, cache.v], 1)
            c2 = bst.KV16Cache(pool[:, 0], pool[:, 1])
        else:
            c2 = bst.KV4Cache(cache.codes, cache.scales.clone())
        V2 = _infinite_values(c2, V.copy(), [int(lists[0, where])])
        some = [0, rows // 2, rows - 1]
        want = [attend_row(_f64(q[r]), K[lists[r]], V2[lists[r]], scale) for r in some]
        assert any(np.isinf(w[0]).any() for w in want)
        vmax = np.abs(V2[np.isfinite(V2)]).max()
        for ws in (bst.attn_workspace("cuda"), None):
            out.fill_(-77.0), lse.fill_(-77.0)
            if window:
                bst.attn_window(q, c2, *[torch.from_numpy(x).cuda() for x in (pt, ptr, pos)], 1, 1 << 20, 0, out[:rows, :hq],
                                scale=scale, lse=lse[:rows], workspace=ws)
            else:
                bst.attn_slots(q, c2, torch.from_numpy(lists).cuda(), out[:rows, :hq], scale=scale, lse=lse[:rows], workspace=ws)
            torch.cuda.synchronize()
            check_rows(_f64(out[some, :hq]), _f64(lse[some]), want, kind, [n] * 3, vmax)

# ---------------------------------------------------------------- small weights

def _attend_counted(q, k, v, times, scale):
    """attend_row over keys of which key i counts times[i] times.  Returns out, lse, A, dx and W, the sum of the weights
    relative to the largest one."""
    hq, d = q.shape
    g = hq // k.shape[1]
    out, lse, A, dx, W = np.zeros((hq, d)), np.zeros(hq), np.zeros((hq, d)), np.zeros(hq), np.zeros(hq)
    for h in range(hq):
        x = scale * (k[:, h // g] @ q[h])
        p = np.exp(x - x.max()) * times
        W[h] = p.sum()
        out[h], A[h] = p @ v[:, h // g] / W[h], p @ np.abs(v[:, h // g]) / W[h]
        lse[h] = x.max() + np.log(W[h])
        S = abs(scale) * (np.abs(k[:, h // g]) @ np.abs(q[h]))
        dx[h] = (d + 16) * 2.0 ** -24 * S.max() + np.abs(x).max() * 2.0 ** -22
    return out, lse, A, dx, W


def _check_counted(got, got_lse, want, kind, n, v):
    """The bounds of attn_ref.py, fp16's term made sharper: a weight is held as
    2^7 times its ratio to the running maximum, which is never above the row's.
    Below 2^-14 that is off by 2^-25 at most, 2^-32 of the largest weight; n such
    errors, in the products (times max |v|) and in the sum (times |out|), over W.
    The output's own rounding below fp16's normal range: 2^-25."""
    u = 2.0 ** -11 if kind == "f16" else 2.0 ** -8
    vmax = np.abs(v).max()
    for r, (out, lse, A, dx, W) in enumerate(want):
        tol = A * (u + 2 * dx[:, None] + 2.0 ** -21 + 2 * n * 2.0 ** -24) + 2 * u * np.abs(out) + 2.0 ** -40
        if kind == "f16":
            tol = tol + 2.0 ** -25 + n * 2.0 ** -32 * (vmax + np.abs(out)) / W[:, None]
        err = np.abs(got[r] - out)
        assert (err <= tol).all(), f"row {r}: worst {(err / tol).max()} tolerances, error {err.max()} of {np.abs(out).max()}"
        el = np.abs(got_lse[r] - lse)
        assert (el <= dx + 2.0 ** -21 + 2 * n * 2.0 ** -24 + np.abs(lse) * 2.0 ** -22).all(), f"row {r}: lse {el.max()}"


def _tail_inputs(form, kind, d, hq, hkv, bits, seed):
    """Two pages of keys whose scores lie about `bits` * ln 2 below that of key 64,
    with values near 1,024 (key 64: 0, so that the result is the others' share).
    Channel 0 makes the distance, in numbers that both types hold exactly; the
    rest is noise."""
    rng = np.random.default_rng(seed)
    k = rng.choice([-0.25, 0.0, 0.25], (128, hkv, d))
    k[:, :, 0] = np.where(np.arange(128) == 64, 4.0, 0.0)[:, None]
    k[:, :, 32:64] = np.round(rng.uniform(-1, 1, (128, hkv, 32)) * 2) / 2
    v = np.where(np.arange(128) == 64, 0.0, 1024.0)[:, None, None] * rng.choice([0.5, 1.0, 1.5], (128, hkv, d))
    q = rng.choice([-1.0, 0.0, 1.0], (1, hq, d)) / 64
    q[:, :, 0] = np.round(bits * np.log(2) / 4 * 32) / 32
    if form == "kv16":
        t = TYPES[kind]
        pool = torch.from_numpy(np.stack([k, v], 1)).to(t).cuda()
        return q, k, v, lambda pages: bst.KV16Cache(pool[:, 0], pool[:, 1])
    c, s = zip(quantise(k), quantise(v))
    kq, vq = (dequantise(a, b) for a, b in zip(c, s))
    cache = bst.KV4Cache(torch.from_numpy(np.stack(c, 2)).cuda(), torch.from_numpy(np.stack(s, 2)).cuda())
    return q, kq, vq, lambda pages: cache


@pytest.mark.parametrize("kind,form,d,hq,hkv", [
    ("f16", "kv16", 64, 8, 2), ("f16", "kv16", 128, 20, 1), ("f16", "kv16", 256, 2, 1), ("f16", "kv4", 64, 4, 4),
    ("f16", "kv4", 128, 16, 2), ("f16", "kv4", 256, 4, 1), ("bf16", "kv16", 128, 8, 1), ("bf16", "kv4", 128, 8, 1)])
@pytest.mark.parametrize("bits,log_n", [(13, 10), (15, 12), (18, 13), (22, 14), (26, 15), (30, 15)])
def test_slots_count_small_weights(kind, form, d, hq, hkv, bits, log_n):
    """A dominating key beside very many whose weights are far below fp16's normal range: their share, of the output
    as of lse, is not lost."""
    say(f"small weights {kind} {form} d={d} hq={hq} bits={bits} n=2^{log_n}")
    q, K, V, make = _tail_inputs(form, kind, d, hq, hkv, bits, d + hq)
    n = (1 << log_n) + 77
    rng = np.random.default_rng(bits)
    lists = rng.integers(0, 64, n).astype(np.int32)
    for at in (0, n // 2, n - 1):
        x = lists.copy()
        x[at] = 64
        times = np.bincount(x, minlength=128)
        want = _attend_counted(q[0], K[:65], V[:65], times[:65], 1.0)
        qd = torch.from_numpy(q).to(TYPES[kind]).cuda()
        out, lse = torch.empty_like(qd), torch.empty((1, hq), dtype=torch.float32, device="cuda")
        for ws in (bst.attn_workspace("cuda"), None):            # split, no wave has all of the tail beside the key
            bst.attn_slots(qd, make(2), torch.from_numpy(x).cuda().view(1, -1), out, scale=1.0, lse=lse, workspace=ws)
            torch.cuda.synchronize()
            _check_counted(_f64(out), _f64(lse), [want], kind, n, V[:65])


@pytest.mark.parametrize("kind,form,d,hq,hkv,rows", [
    ("f16", "kv16", 64, 8, 2, 60), ("f16", "kv16", 128, 8, 1, 70), ("f16", "kv16", 256, 4, 1, 40), ("f16", "kv4", 64, 8, 4, 120),
    ("f16", "kv4", 128, 16, 2, 48), ("f16", "kv4", 256, 4, 1, 3), ("bf16", "kv16", 128, 8, 1, 70), ("f16", "kv16", 128, 8, 1, 1)])
@pytest.mark.parametrize("bits,log_n", [(15, 13), (22, 15), (26, 15), (30, 15)])
def test_windows_count_small_weights(kind, form, d, hq, hkv, rows, bits, log_n):
    """The same through a page table that names the tail's page again and again."""
    say(f"small weights, window {kind} {form} d={d} hq={hq} rows={rows} bits={bits} n=2^{log_n}")
    q, K, V, make = _tail_inputs(form, kind, d, hq, hkv, bits, d + hq)
    pages = (1 << log_n) // 64
    q = np.tile(q, (rows, 1, 1))
    q[:, :, 1:] *= np.random.default_rng(1).choice([-1, 1], (rows, 1, 1))
    qd = torch.from_numpy(q).to(TYPES[kind]).cuda()
    pos = np.arange(pages * 64 - rows, pages * 64, dtype=np.int32) - 64
    some = [0, rows // 2, rows - 1]
    for at in (0, pages // 2, pages - 4):
        pt = np.zeros((1, pages), np.int32)
        pt[0, at] = 1
        times = np.zeros((len(some), 128))
        for i, r in enumerate(some):
            p = np.arange(int(pos[r]) + 1)
            times[i] = np.bincount(pt[0, p // 64] * 64 + p % 64, minlength=128)
        want = [_attend_counted(q[r], K, V, times[i], 1.0) for i, r in enumerate(some)]
        out, lse = torch.empty_like(qd), torch.empty((rows, hq), dtype=torch.float32, device="cuda")
        for ws in (bst.attn_workspace("cuda"), None):
            bst.attn_window(qd, make(2), *[torch.from_numpy(x).cuda() for x in (pt, np.array([0, rows], np.int32), pos)], rows,
                            1 << 40, 0, out, scale=1.0, lse=lse, workspace=ws)
            torch.cuda.synchronize()
            _check_counted(_f64(out[some]), _f64(lse[some]), want, kind, pages * 64, V)


# ---------------------------------------------------------------- scales

@pytest.mark.parametrize("kind,big", [("bf16", 1e18), ("bf16", 1e14), ("f16", 1e3)])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-44, -1e-41, 3e-39, 1e-37])
@pytest.mark.parametrize("rows", [2, 40])
def test_small_scales_of_large_scores(kind, big, scale, rows):
    """Large queries and keys under tiny scales and a scale of 0."""
    say(f"scale {scale} {kind} {big} rows={rows}")
    pt, ptr, pos, pages = _batch([200], [rows], 4)
    cache, K, V = _cache("kv16", kind, pages, 2, 128, 12)
    q, out, lse = _queries(rows, 8, 128, kind, 3)
    pool = torch.stack([cache.k * big, cache.v], 1)
    cache = bst.KV16Cache(pool[:, 0], pool[:, 1])
    q = (q * big).contiguous()
    assert torch.isfinite(q).all() and torch.isfinite(pool).all()
    res, n = _window_want(_f64(q), _f64(cache.k), V, pt, ptr, pos, pages, rows, 70, 3, float(np.float32(scale)))
    args = [torch.from_numpy(x).cuda() for x in (pt, ptr, pos)]
    for wide in (False, True):
        if wide:
            args[0] = torch.nn.functional.pad(args[0], (0, 30000), value=-1)
        bst.attn_window(q, cache, *args, rows, 70, 3, out[:rows, :8], scale=scale, lse=lse[:rows], workspace=bst.attn_workspace("cuda"))
        check_rows(_f64(out[:rows, :8]), _f64(lse[:rows]), res, kind, n, np.abs(V).max())


@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("scale", [2.0 ** 127, -(2.0 ** 127)])
def test_the_largest_scale_of_zero_scores(rows, scale):
    """Queries of zeros weigh all keys alike under any scale that is taken."""
    say(f"scale {scale} rows={rows}")
    pt, ptr, pos, pages = _batch([200], [rows], 4)
    cache, K, V = _cache("kv4", "f16", pages, 2, 128, 12)
    q, out, lse = _queries(rows, 8, 128, "f16", 3)
    q = torch.zeros_like(q).contiguous()
    res, n = _window_want(_f64(q), K, V, pt, ptr, pos, pages, rows, 70, 3, scale)
    args = [torch.from_numpy(x).cuda() for x in (pt, ptr, pos)]
    for wide in (False, True):
        if wide:
            args[0] = torch.nn.functional.pad(args[0], (0, 30000), value=-1)
        bst.attn_window(q, cache, *args, rows, 70, 3, out[:rows, :8], scale=scale, lse=lse[:rows], workspace=bst.attn_workspace("cuda"))
        check_rows(_f64(out[:rows, :8]), _f64(lse[:rows]), res, "f16", n, np.abs(V).max())


# ---------------------------------------------------------------- the path's attention on several streams

def _path(B=2, hi=3000):
    import synth
    from block_scoring_top_amd.pipeline import IndexerPath
    from synth.device import upload
    inp = synth.qsa_verify_64req(B=B, lo=300, hi=hi)
    p = IndexerPath(upload(inp, "cuda"), "decode")
    p.run()
    torch.cuda.synchronize()
    return inp, p


def _spy_on_workspaces(monkeypatch):
    """A list to which every attend() adds its stream and its workspace's address."""
    from block_scoring_top_amd import pipeline
    used, real = [], pipeline.attn_slots

    def spy(*a, workspace, stream, **kw):
        used.append(((stream or torch.cuda.current_stream()).cuda_stream, workspace.data_ptr()))
        return real(*a, workspace=workspace, stream=stream, **kw)

    monkeypatch.setattr(pipeline, "attn_slots", spy)
    return used


def test_attend_on_two_streams_at_once(monkeypatch):
    """Calls on different streams share nothing that they write, whichever comes first; those on one stream need no more
    than one workspace."""
    inp, p = _path()
    say(f"attend on two streams, rows={inp.num_rows}")
    R = inp.num_rows
    cache, _, _ = _cache("kv4", "bf16", inp.num_pages, 2, 128, 11)
    qs = [_queries(R, 16, 128, "bf16", 12 + i)[0].clone() for i in range(2)]
    want = []
    for q in qs:
        o = torch.empty_like(q)
        bst.attn_slots(q, cache, p.slots, o, count=p.out_count, workspace=bst.attn_workspace("cuda"))
        want.append(o)
    used = _spy_on_workspaces(monkeypatch)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(20)] for q in qs]
    torch.cuda.synchronize()
    for k in range(20):
        for i in range(2):
            p.attend(qs[i], cache, outs[i][k], stream=streams[i])
    torch.cuda.synchronize()
    assert len({s for s, _ in used}) == 2 and len(set(used)) == 2 and len({w for _, w in used}) == 2
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, want[i])


def test_captured_attends_share_no_workspace(monkeypatch):
    """Two graphs captured from one path, replayed at once on two streams and beside eager calls."""
    inp, p = _path()
    say(f"captured attends, rows={inp.num_rows}")
    R = inp.num_rows
    cache, _, _ = _cache("kv4", "bf16", inp.num_pages, 2, 128, 11)
    qs = [torch.empty((R, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    outs = [torch.empty_like(q) for q in qs]
    p.attend(qs[0].normal_(generator=torch.Generator(device="cuda").manual_seed(1)), cache, outs[0])
    graphs, seen = [], []
    used = _spy_on_workspaces(monkeypatch)
    p.attend(qs[0], cache, outs[0])
    seen.append({w for _, w in used})
    for i in range(2):
        used.clear()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.attend(qs[i], cache, outs[i])
            p.attend(qs[i], cache, outs[i])                      # as of two layers: they may share
        graphs.append(g)
        seen.append({w for _, w in used})
    assert not (seen[0] & seen[1] or seen[0] & seen[2] or seen[1] & seen[2])
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = bst.attn_workspace("cuda")
    for rep in range(6):
        want = []
        for i, q in enumerate(qs):
            q.copy_(torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(10 * rep + i), device="cuda"))
            o = torch.empty_like(q)
            bst.attn_slots(q, cache, p.slots, o, count=p.out_count, workspace=ws)
            want.append(o)
            outs[i].fill_(-77.0)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                for _ in range(4):
                    g.replay()
        for _ in range(8):
            p.attend(qs[2], cache, outs[2])
        torch.cuda.synchronize()
        for i in range(3):
            assert torch.equal(outs[i], want[i]), (rep, i)


# ---------------------------------------------------------------- very large scores

@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 4, 4), (128, 20, 1), (256, 4, 1)])
@pytest.mark.parametrize("kind,form,bits", [("bf16", "kv16", b) for b in (3, 20, 24, 27, 31, 40, 90)] +
                         [("f16", "kv16", b) for b in (3, 18, 23, 25)] + [("bf16", "kv4", b) for b in (3, 24, 31, 100)] +
                         [("f16", "kv4", b) for b in (3, 17, 23, 26)])
@pytest.mark.parametrize("rows", [1, 6, 70])
@pytest.mark.parametrize("scale", [1.0, 0.7, -1.7])
def test_very_large_scores(kind, form, bits, d, hq, hkv, rows, scale):
    """Products of small whole numbers times 2^bits, exact in FP32: keys with the best of them share a row's result. The
    scales make their products with log2(e) be rounded up, down and not at all."""
    say(f"scores of 2^{bits} {kind} {form} d={d} hq={hq} rows={rows} scale={scale}")
    rng = np.random.default_rng(bits + d)
    ctx = [300]
    pt, ptr, pos, pages = _batch(ctx, [rows], 8)
    c = rng.integers(-6, 3, (pages * 64, hkv))
    at = pt[0, np.arange(300) // 64] * 64 + np.arange(300) % 64
    c[at[[5, 37, 100, 229]]] = 3                                 # the best: equal, in different steps of the kernels
    c[at[10:30]] = -6
    c = np.where(c == 3, 6, np.where(np.abs(c) == 5, 4, c)).astype(np.float64)    # numbers of the 4-bit form
    v = rng.choice([-6, -4, -3, -2, -1.5, -1, -.5, .5, 1, 1.5, 2, 3, 4, 6], (pages * 64, hkv, d))
    k = np.zeros((pages * 64, hkv, d))
    k[:, :, 7] = c
    half = bits // 2
    q = np.zeros((rows, hq, d))
    q[:, :, 7] = np.copysign(2.0 ** (bits - half), scale)
    scale = float(np.float32(scale))
    if form == "kv16":
        pool = torch.from_numpy(np.stack([k * 2.0 ** half, v], 1)).to(TYPES[kind]).cuda()
        cache = bst.KV16Cache(pool[:, 0], pool[:, 1])
    else:
        mag = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
        codes = lambda x: (np.abs(np.abs(x)[..., None] - mag).argmin(-1) + 8 * (x < 0)).astype(np.uint8)  # noqa: E731
        pack = lambda x: x[..., 0::2] | x[..., 1::2] << 4  # noqa: E731
        s = np.full((pages * 64, hkv, 2, d // 32), 127, np.uint8)
        s[:, :, 0] += np.uint8(half)
        cache = bst.KV4Cache(torch.from_numpy(np.stack([pack(codes(k)), pack(codes(v))], 2)).cuda(), torch.from_numpy(s).cuda())
    qd = torch.from_numpy(q).to(TYPES[kind]).cuda()
    assert np.array_equal(_f64(qd), q)
    u = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    out, lse = torch.empty_like(qd), torch.empty((rows, hq), dtype=torch.float32, device="cuda")
    args = [torch.from_numpy(x).cuda() for x in (pt, ptr, pos)]
    for wide in (False, True):
        if wide:
            args[0] = torch.nn.functional.pad(args[0], (0, 30000), value=-1)
        for ws in (bst.attn_workspace("cuda"), None):
            out.fill_(-77.0), lse.fill_(-77.0)
            bst.attn_window(qd, cache, *args, rows, 1 << 40, 0, out, scale=scale, lse=lse, workspace=ws)
            torch.cuda.synchronize()
            for r in {0, rows // 2, rows - 1}:
                seen = at[:int(pos[r]) + 1]
                for h in range(hq):
                    g = h // (hq // hkv)
                    x = c[seen, g] * 2.0 ** bits * abs(scale)
                    w = np.exp(x - x.max())
                    want = w @ v[seen, g] / w.sum()
                    wl = x.max() + np.log(w.sum())
                    tol = (w @ np.abs(v[seen, g]) / w.sum()) * (u + 2.0 ** -10) + 2 * u * np.abs(want)
                    got = _f64(out[r, h])
                    assert (np.abs(got - want) <= tol).all(), (r, h, got[:4], want[:4])
                    assert abs(float(lse[r, h]) - wl) <= abs(wl) * 2.0 ** -20 + 2.0 ** -12, (r, h, float(lse[r, h]), wl)


# ---------------------------------------------------------------- the 4-bit cache over its whole range

@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_every_scale_and_code_reads_back(kind):
    """Every code with every scale byte, those that kv4_store does not write (0 .. 6, 253, 254) among them, in each type,
    rounded once."""
    say(f"kv4_load of every scale {kind}")
    scales = np.arange(256).astype(np.uint8)
    n = len(scales)
    codes = np.zeros((n, 1, 2, 32), np.uint8)
    codes[..., :16] = np.arange(8)[[0, 1, 2, 3, 4, 5, 6, 7] * 2] * 2 % 16 | (np.arange(16) << 4) & 0xF0
    codes[..., 16:] = np.arange(16) | (15 - np.arange(16)) << 4
    sc = np.full((n, 1, 2, 2), 127, np.uint8)
    sc[:] = scales[:, None, None, None]
    cache = bst.KV4Cache(torch.from_numpy(codes).cuda(), torch.from_numpy(sc).cuda())
    k, v = (torch.empty((n, 1, 64), dtype=TYPES[kind], device="cuda") for _ in range(2))
    bst.kv4_load(cache, torch.arange(n, dtype=torch.int32, device="cuda"), k, v)
    want = torch.from_numpy(dequantise(codes, sc)).to(TYPES[kind])
    for i, got in enumerate((k, v)):
        np.testing.assert_array_equal(_f64(got), _f64(want[:, :, i]))


@pytest.mark.parametrize("rows", [1, 6, 150])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 8, 1), (256, 4, 1)])
@pytest.mark.parametrize("window", [40, 1 << 30])
def test_fp16_over_large_and_small_scales(rows, d, hq, hkv, window):
    """4-bit values past fp16's range are infinities to fp16 queries (in V: K stays in it), those below it are rounded; where
    a row does not see them they do not reach it."""
    say(f"fp16 over large and small scales rows={rows} d={d} window={window}")
    pt, ptr, pos, pages = _batch([200], [rows], 8)
    cache, K, V = _cache("kv4", "f16", pages, hkv, d, 41)
    rng = np.random.default_rng(5)
    scales = cache.scales.cpu().numpy()
    scales[:, :, 1] = rng.integers(127 - 26, 127 + 12, scales[:, :, 1].shape)    # 2^-26 .. 2^11
    scales[:, :, 0, 0] -= 8                                                       # small keys in one group
    for p in (199, 198, 130, 90, 20):
        s = int(pt[0, p // 64]) * 64 + p % 64
        scales[s, :, 1] = rng.integers(127 + 13, 127 + 18, scales[s, :, 1].shape)   # from 2^13: 6 * 2^14 is past the range
    cache = bst.KV4Cache(cache.codes, torch.from_numpy(scales).cuda())
    kv = torch.from_numpy(dequantise(cache.codes.cpu().numpy(), scales)).to(torch.float16).double().numpy()
    K, V = kv[:, :, 0], kv[:, :, 1]
    q, out, lse = _queries(rows, hq, d, "f16", 2)
    res, n = _window_want(_f64(q), K, V, pt, ptr, pos, pages, rows, window, 4, 0.09)
    assert any(np.isinf(r[0]).any() for r in res)
    args = [torch.from_numpy(x).cuda() for x in (pt, ptr, pos)]
    for wide in (False, True):                                   # a wide page table: the prefill kernel, its pages split
        if wide:
            args[0] = torch.nn.functional.pad(args[0], (0, 30000), value=-1)
        for ws in (bst.attn_workspace("cuda"), None):
            out.fill_(-77.0), lse.fill_(-77.0)
            bst.attn_window(q, cache, *args, rows, window, 4, out[:rows, :hq], scale=0.09, lse=lse[:rows], workspace=ws)
            torch.cuda.synchronize()
            check_rows(_f64(out[:rows, :hq]), _f64(lse[:rows]), res, "f16", n, np.abs(V[np.isfinite(V)]).max())


# ---------------------------------------------------------------- the largest launches

def _one_key_cache(kind, form):
    """Two pages of one head of 64 whose values both forms hold exactly."""
    k = torch.randint(-6, 7, (128, 1, 64), generator=_gen(1), device="cuda")
    v = torch.randint(-3, 4, (128, 1, 64), generator=_gen(2), device="cuda")
    pool = torch.stack([k, v], 1).to(TYPES[kind])
    if form == "kv16":
        return bst.KV16Cache(pool[:, 0], pool[:, 1]), pool[:, 1]
    cache = bst.KV4Cache.empty(2, 1, 64, "cuda")
    bst.kv4_store(pool[:, 0].contiguous(), pool[:, 1].contiguous(), torch.arange(128, dtype=torch.int32, device="cuda"), cache)
    return cache, pool[:, 1]


@pytest.mark.parametrize("form", ["kv4", "kv16"])
def test_two_million_rows_of_one_key(form):
    """The most row tiles that a call takes (2^21), by lists and by windows: each row is the value of its one key."""
    n = 1 << 21
    say(f"2^21 rows {form}")
    cache, v = _one_key_cache("bf16", form)
    q = torch.randn((n, 1, 64), generator=_gen(3), device="cuda").bfloat16()
    at = torch.randint(-1, 128, (n,), generator=_gen(4), device="cuda", dtype=torch.int32)
    want = torch.where((at >= 0)[:, None, None], v[at.clamp(min=0).long()], 0)
    out = torch.full_like(q, -77.0)
    bst.attn_slots(q, cache, at.view(-1, 1), out, workspace=bst.attn_workspace("cuda"))
    assert torch.equal(out, want)
    out.fill_(-77.0)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda").repeat(n, 1)
    ptr = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    want = torch.where((at >= 0)[:, None, None], v[(at.clamp(min=0).long() + 64) % 128], 0)
    bst.attn_window(q, cache, table, ptr, at, 1, 1, 0, out, workspace=bst.attn_workspace("cuda"))
    assert torch.equal(out, want)
    with pytest.raises(bst.BlockScoreError):
        q2 = torch.empty((n + 1, 1, 64), dtype=torch.bfloat16, device="cuda")
        bst.attn_slots(q2, cache, torch.zeros((n + 1, 1), dtype=torch.int32, device="cuda"), torch.empty_like(q2))


@pytest.mark.parametrize("form", ["kv4", "kv16"])
def test_a_million_requests_in_the_prefill_kernel(form):
    """2^20 requests of up to 300 rows (two tiles each, the most that the prefill kernel takes), three of which have any."""
    n = 1 << 20
    say(f"2^20 requests {form}")
    cache, v = _one_key_cache("bf16", form)
    counts = torch.zeros(n, dtype=torch.int64, device="cuda")
    counts[0], counts[n // 2 + 3], counts[n - 1] = 300, 257, 1
    ptr = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int()
    rows = int(counts.sum())
    q = torch.randn((rows, 1, 64), generator=_gen(3), device="cuda").bfloat16()
    at = torch.randint(-1, 128, (rows,), generator=_gen(4), device="cuda", dtype=torch.int32)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda").repeat(n, 1)
    want = torch.where((at >= 0)[:, None, None], v[(at.clamp(min=0).long() + 64) % 128], 0)
    out = torch.full_like(q, -77.0)
    bst.attn_window(q, cache, table, ptr, at, 300, 1, 0, out, workspace=bst.attn_workspace("cuda"))
    assert torch.equal(out, want)


def test_store_and_load_of_more_pieces_than_a_launch_takes():
    """16,500 rows x 8,192 heads of 64: 2^31 pieces of 8 channels and some, in two launches each."""
    T, hkv, d = 16500, 8192, 64
    say("kv4 of more than 2^31 pieces")
    x = torch.empty((T, hkv, d), dtype=torch.float16, device="cuda").normal_(generator=_gen(1))
    pages = -(-T // 64)
    cache = bst.KV4Cache(torch.empty((pages * 64, hkv, 2, 32), dtype=torch.uint8, device="cuda"),
                         torch.empty((pages * 64, hkv, 2, 2), dtype=torch.uint8, device="cuda"))
    slots = (T - 1 - torch.arange(T, device="cuda")).int()
    bst.kv4_store(x, x, slots, cache)
    some = [0, 1, 16382, 16383, 16384, 16385, T - 1]
    for i in some:
        c, s = quantise(_f64(x[i]))
        for which in range(2):
            np.testing.assert_array_equal(cache.codes[T - 1 - i, :, which].cpu().numpy(), c)
            np.testing.assert_array_equal(cache.scales[T - 1 - i, :, which].cpu().numpy(), s)
    y = torch.zeros_like(x)
    bst.kv4_load(cache, slots, y, x)                             # K into y, V over the input
    assert torch.equal(x, y)
    for i in some:
        np.testing.assert_array_equal(_f64(y[i]), dequantise(cache.codes[T - 1 - i, :, 0].cpu().numpy(),
                                                             cache.scales[T - 1 - i, :, 0].cpu().numpy()))
    del x, y, cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("form", ["kv4", "kv16"])
def test_a_list_of_almost_2_to_the_31_entries(form):
    """Counts within a step of 2^31: the entries are -1 but for some at the front, in the middle and at the end."""
    say(f"a list of 2^31 - 1 entries {form}")
    n = 2**31 - 1
    cache, K, V = _cache(form, "bf16", 4, 1, 128, 3)
    at = np.r_[np.arange(40), 2**30 + np.arange(70), n - 33 + np.arange(33)]
    slots = np.random.default_rng(2).integers(0, 256, len(at)).astype(np.int32)
    lists = torch.full((1, n), -1, dtype=torch.int32, device="cuda")
    lists[0, torch.from_numpy(at).cuda()] = torch.from_numpy(slots).cuda()
    q, out, lse = _queries(1, 4, 128, "bf16", 4)
    ws = bst.attn_workspace("cuda")
    for count in (n, n - 1, n - 32, None):
        s = slots if count is None else slots[at < count]
        want = attend_row(_f64(q[0]), K[s], V[s], 128 ** -0.5)
        c = None if count is None else torch.tensor([count], dtype=torch.int32, device="cuda")
        bst.attn_slots(q, cache, lists, out[:1, :4], count=c, lse=lse[:1], workspace=ws)
        torch.cuda.synchronize()
        check_rows(_f64(out[:1, :4]), _f64(lse[:1]), [want], "bf16", [len(s)], np.abs(V).max())
    del lists
    torch.cuda.empty_cache()


def test_lists_wider_than_32_bits_are_refused():
    """2^32 + 3 entries a row are not taken for 3."""
    say("lists of 2^32 + 3 entries")
    cache, _ = _one_key_cache("bf16", "kv4")
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    lists = torch.empty((1, 2**32 + 3), dtype=torch.int32, device="cuda")
    lists[0, :3] = -1
    with pytest.raises(ValueError, match="2\\^31"):
        bst.attn_slots(q, cache, lists, torch.empty_like(q))
    with pytest.raises(ValueError, match="2\\^31"):
        bst.prepare_attn_slots(q, cache, lists, torch.empty_like(q))
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        bst.attn_window(q, cache, lists, one, one[:1], 1, 1, 0, torch.empty_like(q))
    del lists
    torch.cuda.empty_cache()
