"""Cases, plain forms and 64-bit values of the batch's page tables, the 8-bit KV cache and the 4-bit index keys.

``pages_extend`` and ``pages_release`` keep the page tables of a batch on the
GPU: pages for the new tokens, row positions, slots, and pages given back.
``kv8_store`` quantises K/V rows into a paged cache of E4M3 codes with one
power-of-two scale per page (64 tokens), kv head and K or V; ``kv8_load`` reads
rows back; ``attn_slots`` and ``attn_window`` attend over it.  ``idx4_store``
and ``idx4_compress_store`` write the indexer's keys as E2M1 codes with a
power-of-two scale per 32 channels (``idx4_load`` reads them back), and
``idx4_score`` scores 4-bit queries against them.

``run`` computes the plain form in elementary torch operations in 32 bits, or,
where ``own`` is true, makes the framework's calls.
"""
import math

import torch

own = False

PAGE = 64
GROUP = 32
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
DEV = "cuda"
KV8_EMIN, KV8_EMAX, KV8_TOP = -120, 119, 448.0      # exponents of a page's scale, largest E4M3 value
FP4_EMIN, FP4_EMAX = -120, 125                      # exponents of a group's scale
IDX_HEADS, IDX_DIM, ROTARY, SECTIONS, THETA = 4, 128, 128, (16, 24, 24), 1e6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the tables of a verify step: 64 requests of 4K to 131K tokens, 6 drafted rows each, rejected ones given back
        dict(name="pages_verify_64x6", op="pages", req=64, lo=4096, hi=131072, new=6, prompts=0, prompt=0, pad=0),
        # a mixed step of 1,003 requests: most decode, 13 bring prompt chunks of up to 8,192 tokens; padded rows
        dict(name="pages_mixed_1003", op="pages", req=1003, lo=200, hi=60000, new=1, prompts=13, prompt=8192, pad=77),
        # one new token of each of 64 requests appended to pages that hold earlier ones: latency counts
        dict(name="kv8_decode_64", op="kv8", req=64, rows=1, hkv=2, d=128, type="bf16", fused=True, pad=0),
        # a prefill chunk that starts inside a page
        dict(name="kv8_prefill_8k", op="kv8", req=1, rows=8192, hkv=8, d=128, type="bf16", fused=False, pad=0),
        # one decode row at 8,192 tokens + 2 pending, c = 4, top-512
        dict(name="slots8_decode_1x8k", op="slots", req=1, rows=1, lo=8194, hi=8194, c=4, k=512, hq=16, hkv=2, d=128,
             type="bf16"),
        # speculative verify: 64 requests of 4K to 131K tokens, 6 rows each, c = 4, top-512
        dict(name="slots8_verify_64x6", op="slots", req=64, rows=6, lo=4096, hi=131072, c=4, k=512, hq=16, hkv=2,
             d=128, type="bf16"),
        # an odd ragged batch: 5 requests of 301 to 1,505 rows, odd window, fp16
        dict(name="window8_ragged_5", op="window", req=5, rows=1505, lo=1600, hi=20001, window=1021, sinks=13, hq=12,
             hkv=4, d=128, type="f16"),
        # an 8,192-row prefill chunk of a 64K context
        dict(name="window8_prefill_8k", op="window", req=1, rows=8192, lo=65536, hi=65536, window=4096, sinks=4, hq=16,
             hkv=2, d=128, type="bf16"),
        # the index keys (c = 1) of one new token of each of 64 requests: latency counts
        dict(name="idx4_store_64", op="keys", c=1, req=64, rows=1, type="bf16", pad=0),
        # the raw index keys of an 8,192-token prefill chunk, compressed by 4
        dict(name="idx4_compress_8k", op="keys", c=4, req=1, rows=8192, type="bf16", pad=0),
        # 16 decode rows at 81,920 tokens, c = 1
        dict(name="score4_16x80k", op="score", req=16, rows=1, lo=81920, hi=81920, c=1),
        # an 8,192-row prefill chunk of a 64K context, c = 4
        dict(name="score4_prefill_8k", op="score", req=1, rows=8192, lo=65536, hi=65536, c=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "kv8", "slots", "window", "keys", "score"])
    hi = _log(rng, 600, 100000)
    lo = max(64, int(hi * rng.uniform(0.1, 1)))
    if op == "pages":
        req = _log(rng, 1, 1003)
        prompts = rng.choice([0, 0, rng.randint(1, min(13, req))])
        return dict(op=op, req=req, lo=lo, hi=hi, new=rng.choice([1, 6, rng.randint(0, 70)]), prompts=prompts,
                    prompt=_log(rng, 64, 8192) if prompts else 0, pad=rng.randint(0, 100))
    hkv = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    if op == "kv8":
        rows = rng.choice([1, 6, _log(rng, 7, 2048)])
        req = _log(rng, 1, 200 if rows <= 6 else 4)
        return dict(op=op, req=req, rows=rows, hkv=hkv, d=min(d, 1024 // hkv), type=rng.choice(["bf16", "f16", "f32"]),
                    fused=rng.random() < 0.5, pad=rng.randint(0, max(0, req * rows // 50)))
    if op == "keys":
        rows = rng.choice([1, 6, _log(rng, 7, 2048)])
        c = rng.choice([1, 4])
        return dict(op=op, c=c, req=_log(rng, 1, 200 if rows <= 6 else 4), rows=rows,
                    type="bf16" if c == 4 else rng.choice(["bf16", "f16", "f32"]), pad=rng.randint(0, 5) if c == 1 else 0)
    if op == "score":
        rows = rng.choice([1, 1, 2, 6, _log(rng, 20, 2000)])
        req = _log(rng, 1, 64) if rows <= 6 else rng.randint(1, 3)
        while req * hi > 16 * 81920 and req > 1:
            req //= 2
        return dict(op=op, req=req, rows=min(rows, lo), lo=lo, hi=hi, c=rng.choice([1, 4]))
    group = rng.choice([1, 4, 7, 8])
    kind = rng.choice(["bf16", "bf16", "f16"])
    if op == "slots":
        c = rng.choice([1, 4])
        k = _log(rng, 16, 512) if c == 4 else _log(rng, 64, 2048)
        rows = rng.choice([1, 1, 1, 2, 6, _log(rng, 32, 512)])
        req = 1 if rows > 6 else _log(rng, 1, 48)
        # at most what the verify case reads: 384 rows x 2,051 slots x 2 heads of 128
        while req * rows * c * k * hkv * d > 384 * 2051 * 2 * 128 and max(req, rows) > 1:
            req, rows = (req // 2, rows) if req > 1 else (req, rows // 2)
        while req * hi * hkv * d > 16 * 81920 * 4 * 128 and req > 1:
            req //= 2
        return dict(op=op, req=req, rows=min(rows, lo), lo=lo, hi=hi, c=c, k=k, hq=hkv * group, hkv=hkv, d=d, type=kind)
    window, sinks = _log(rng, 16, 4096), rng.choice([0, 1, 4, rng.randint(5, 100)])
    rows = rng.choice([1, 1, 6, _log(rng, 50, 2000)])
    req = _log(rng, 1, 48) if rows <= 6 else rng.randint(1, 3)
    hkv = min(hkv, 4)
    while req * hi * hkv * d > 16 * 81920 * 4 * 128 and req > 1:
        req //= 2
    while req * rows * (window + rows) * hkv * group * d > 8192 * 8192 * 16 * 128 // 2 and rows > 1:
        rows //= 2
    return dict(op=op, req=req, rows=min(rows, lo), lo=lo, hi=hi, window=window, sinks=sinks, hq=hkv * group, hkv=hkv,
                d=d, type=kind)


def _contexts(case):
    """Tokens of each request, spread evenly over the logarithm of lo .. hi."""
    n, lo, hi = case["req"], case["lo"], case["hi"]
    return [int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]


def _row_counts(case):
    """Query rows of each request: all alike, or (prefill of several requests) growing to `rows`."""
    n, rows = case["req"], case["rows"]
    return [rows if rows <= 6 else max(1, rows * (i + 1) // n) for i in range(n)]


def _new_counts(case):
    """New tokens of each request of a step: `new`, but a prompt chunk of up to `prompt` for `prompts` of them."""
    n = [case["new"]] * case["req"]
    for i in range(case["prompts"]):
        n[(2 * i + 1) * case["req"] // (2 * case["prompts"])] = max(1, case["prompt"] * (i + 1) // case["prompts"])
    return n


def _offsets(case):
    """Where in its page each request's first new token lies (chunks that are compressed start with a block of 4)."""
    at = [(37 * b + 11) % PAGE for b in range(case["req"])]
    return [o // 4 * 4 for o in at] if case.get("c") == 4 and case["rows"] > 1 else at


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _rows(g, n, heads, d, spread=0.6):
    """Keys or values: normal, with channels of different size as projections give them."""
    x = torch.randn((n, heads, d), generator=g, device=DEV)
    return x * torch.exp(spread * torch.randn((1, heads, d), generator=g, device=DEV))


def _layout(case, g):
    """page_table [B, stride], req_row_ptr, row_pos, pages in the pool: each request's pages at random places."""
    ctx, rows = _contexts(case), _row_counts(case)
    pages = [-(-t // PAGE) for t in ctx]
    perm = torch.randperm(sum(pages), generator=g, device=DEV, dtype=torch.int32)
    table = torch.full((len(ctx), max(pages)), -1, dtype=torch.int32, device=DEV)
    ptr, pos, at = [0], [], 0
    for b, (t, n, p) in enumerate(zip(ctx, rows, pages)):
        table[b, :p] = perm[at:at + p]
        at += p
        ptr.append(ptr[-1] + n)
        pos.append(torch.arange(t - n, t, dtype=torch.int32, device=DEV))
    return table, _int(ptr), torch.cat(pos), sum(pages)


def _prepare_pages(case, g):
    ctx, new = _contexts(case), _new_counts(case)
    held = [-(-t // PAGE) for t in ctx]
    want = sum(-(-(t + n) // PAGE) - h for t, n, h in zip(ctx, new, held))
    used = sum(held)
    perm = torch.randperm(used + want + 40, generator=g, device=DEV, dtype=torch.int32)
    stride = max(-(-(t + n) // PAGE) for t, n in zip(ctx, new)) + 3
    table = torch.full((len(ctx), stride), -1, dtype=torch.int32, device=DEV)
    ids, at = perm.tolist(), 0
    rows = [ids[a:a + h] + [-1] * (stride - h) for a, h in zip([sum(held[:b]) for b in range(len(held))], held)]
    table.copy_(_int(rows))
    # the ring of free pages starts somewhere in the middle
    size, free = used + want + 40, want + 40
    head = size - free // 2
    ring = torch.zeros(size, dtype=torch.int32, device=DEV)
    ring[(head + torch.arange(free, device=DEV)) % size] = perm[used:]
    kept = [t + (n if n <= 1 else 1 + int(x * n)) for t, n, x in zip(ctx, new, torch.rand(
        len(ctx), generator=g, device=DEV).tolist())]
    total = sum(new) + case["pad"]
    n = dict(dtype=torch.int32, device=DEV)
    return dict(kv_len=_int(ctx), held=_int(held), new_len=_int(new), keep_len=_int(kept), table=table, ring=ring,
                pool=_int([head, free, 0, 0]), ptr=torch.empty(len(ctx) + 1, **n), pos=torch.empty(total, **n),
                slots=torch.empty(total, **n),
                mid=[torch.empty(len(ctx), **n), torch.empty(len(ctx), **n), torch.zeros(4, **n)],
                end=[torch.empty(len(ctx), **n), torch.empty(len(ctx), **n), torch.zeros(4, **n)])


def _new_slots(case, g):
    """Slots of the new tokens (-1 for padding), the filled slots of the pages that they touch, the pool's pages, and
    the page table of the touched pages."""
    off, n = _offsets(case), case["rows"]
    pages = [-(-(o + n) // PAGE) for o in off]
    perm = torch.randperm(sum(pages) + 5, generator=g, device=DEV, dtype=torch.int32)
    width = max(pages)
    table = torch.full((case["req"], width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = perm[at:at + p]
        at += p
    every = (table[:, :, None] * PAGE + torch.arange(PAGE, device=DEV, dtype=torch.int32)).flatten(1)
    p = torch.arange(width * PAGE, device=DEV)
    o = torch.tensor(off, device=DEV)[:, None]
    new = every[(p >= o) & (p < o + n)]
    look = every[p < o + n]
    pad = torch.full((case.get("pad", 0),), -1, dtype=torch.int32, device=DEV)
    return torch.cat([new, pad]).contiguous(), look.contiguous(), sum(pages) + 5, table, every, (p < o)


def _prepare_kv8(case, g):
    hkv, d, kind = case["hkv"], case["d"], TYPES[case["type"]]
    slots, look, pages, _, every, old = _new_slots(case, g)
    n = slots.shape[0]
    s = dict(slots=slots, look=look)
    if case["fused"]:  # K and V as they lie in the output of a fused q/k/v projection
        qkv = torch.cat([_rows(g, n, 2 * hkv, d), _rows(g, n, 2 * hkv, d)], 1).to(kind)
        s["k"], s["v"] = qkv[:, 2 * hkv:3 * hkv], qkv[:, 3 * hkv:]
    else:
        s["k"], s["v"] = (_rows(g, n, hkv, d).to(kind) for _ in range(2))
    # the earlier tokens of the first pages, some pages of them smaller than what is to come
    k, v = (_rows(g, pages * PAGE, hkv, d) for _ in range(2))
    size = torch.exp(0.7 * torch.randn((pages, 1, 1, 1), generator=g, device=DEV))
    there = torch.zeros(pages * PAGE, device=DEV)
    there[every[old].long()] = 1.0
    k, v = ((x.unflatten(0, (pages, PAGE)) * size).flatten(0, 1) * there[:, None, None] for x in (k, v))
    s["codes"], s["scales"] = _pool8(k, v)
    s["k_out"], s["v_out"] = (torch.empty((look.shape[0], hkv, d), dtype=kind, device=DEV) for _ in range(2))
    return s


def _prepare_keys(case, g):
    c = case["c"]
    slots, _, pages, table, _, _ = _new_slots(case, g)
    n = slots.shape[0]
    s = dict(codes=torch.zeros((pages * PAGE // c, IDX_DIM // 2), dtype=torch.uint8, device=DEV),
             scales=torch.full((pages * PAGE // c, IDX_DIM // GROUP), 127, dtype=torch.uint8, device=DEV))
    s["keys"] = _rows(g, n, 1, IDX_DIM)[:, 0].to(TYPES[case["type"]]).contiguous()
    if c == 1:
        s["slots"] = slots
        s["look"] = slots
    else:
        off, rows, req = _offsets(case), case["rows"], case["req"]
        s["ptr"] = _int([rows * b for b in range(req + 1)])
        s["start"] = _int(off)
        s["ring"] = torch.randn((req, 4, IDX_DIM), generator=g, device=DEV).to(torch.bfloat16)
        s["table"] = table
        # every block that the call completes
        at = [(b, j) for b, o in enumerate(off) for j in range(o // 4, (o + rows) // 4)]
        s["blocks"] = torch.tensor(at, dtype=torch.int64, device=DEV).reshape(-1, 2)
        b, j = s["blocks"][:, 0], s["blocks"][:, 1]
        s["look"] = (table[b, j // (PAGE // 4)] * (PAGE // 4) + j % (PAGE // 4)).int().contiguous()
    s["out"] = torch.empty((s["look"].shape[0], IDX_DIM), dtype=torch.float32, device=DEV)
    return s


def _prepare_score(case, g):
    c = case["c"]
    s = {}
    s["table"], s["ptr"], s["pos"], pages = _layout(case, g)
    rows = s["pos"].shape[0]
    s["q"] = torch.randn((rows, IDX_HEADS, IDX_DIM), generator=g, device=DEV).to(torch.bfloat16)
    k = torch.randn((pages * PAGE // c, IDX_DIM), generator=g, device=DEV)
    s["codes"], s["scales"] = _quantise4(k / k.norm(dim=1, keepdim=True))
    s["max_vis"] = max(_contexts(case)) // c
    s["scores"] = torch.zeros((rows, (s["max_vis"] + 3) // 4 * 4), dtype=torch.float32, device=DEV)
    s["len"] = torch.empty(rows, dtype=torch.int32, device=DEV)
    return s


def _prepare_attn(case, g):
    hkv, d, kind = case["hkv"], case["d"], TYPES[case["type"]]
    s = dict(case=case)
    s["table"], s["ptr"], s["pos"], pages = _layout(case, g)
    s["codes"], s["scales"] = _pool8(*(_rows(g, pages * PAGE, hkv, d) for _ in range(2)))
    rows, hq = s["pos"].shape[0], case["hq"]
    s["q"] = (1.2 * torch.randn((rows, hq, d), generator=g, device=DEV)).to(kind)
    s["out"] = torch.empty((rows, hq, d), dtype=kind, device=DEV)
    s["lse"] = torch.empty((rows, hq), dtype=torch.float32, device=DEV)
    if case["op"] == "slots":
        s["slots"], s["count"] = _selection(case, s, g)
    return s


def _selection(case, s, g):
    """The slot list of each row as the selection leaves it: min(k, visible) blocks of c tokens chosen at random,
    the pending tokens, -1 behind them; and the counts."""
    c, k, table = case["c"], case["k"], s["table"].long()
    pos = s["pos"].long()
    rows = pos.shape[0]
    req = torch.bucketize(torch.arange(rows, device=DEV), s["ptr"][1:-1].long(), right=True)
    vis = (pos + 1) // c
    n = int(case["hi"]) // c + 1
    order = torch.rand((rows, n), generator=g, device=DEV)
    order = torch.where(torch.arange(n, device=DEV) < vis[:, None], order, -1.0)
    best = order.topk(min(k, n), dim=1)
    block = torch.where(best.values >= 0, best.indices, -1)
    p = torch.where(block[..., None] >= 0, block[..., None] * c + torch.arange(c, device=DEV), -1).flatten(1)
    taken = torch.clamp(vis, max=min(k, n)) * c
    width = k * c + c - 1
    full = torch.full((rows, width), -1, dtype=torch.int64, device=DEV)
    full[:, :p.shape[1]] = p
    i = torch.arange(width, device=DEV)
    tail = vis[:, None] * c + (i - taken[:, None])
    full = torch.where((i >= taken[:, None]) & (tail <= pos[:, None]), tail, full)
    full = torch.where((i >= taken[:, None]) & (tail > pos[:, None]), -1, full)
    page = torch.gather(table[req], 1, full.clamp(min=0) // PAGE)
    slots = torch.where(full >= 0, page * PAGE + full % PAGE, -1).int()
    return slots, (slots >= 0).sum(1).int()


_PREPARE = {"pages": _prepare_pages, "kv8": _prepare_kv8, "keys": _prepare_keys, "score": _prepare_score,
            "slots": _prepare_attn, "window": _prepare_attn}


def prepare(case, seed):
    s = _PREPARE[case["op"]](case, _gen(seed))
    s["case"] = case
    if own:
        s["calls"] = _own_calls(s)
    return s


# ---------------------------------------------------------------- the framework's calls

def _own_calls(s):
    """The framework's calls with their arguments marshalled once, as a serving loop over fixed buffers keeps them."""
    import block_scoring_top_amd as bst

    case = s["case"]
    op = case["op"]
    if op == "pages":
        pool = bst.PagePool(s["ring"], s["pool"])
        mid, end = (bst.PagePool(s["ring"], s[n][2]) for n in ("mid", "end"))
        return [bst.prepare_pages_extend(pool, s["kv_len"], s["held"], s["new_len"], s["table"], s["ptr"], s["pos"],
                                         s["slots"], kv_len_out=s["mid"][0], held_out=s["mid"][1], pool_out=mid),
                bst.prepare_pages_release(mid, s["mid"][0], s["mid"][1], s["keep_len"], s["table"],
                                          kv_len_out=s["end"][0], held_out=s["end"][1], pool_out=end)]
    if op == "kv8":
        cache = bst.KV8Cache(s["codes"], s["scales"])
        return [bst.prepare_kv8_store(s["k"], s["v"], s["slots"], cache),
                bst.prepare_kv8_load(cache, s["look"], s["k_out"], s["v_out"])]
    if op in ("keys", "score"):
        cache = bst.Idx4Cache(s["codes"], s["scales"], case["c"])
    if op == "keys":
        if case["c"] == 1:
            store = bst.prepare_idx4_store(s["keys"], s["slots"], cache)
        else:
            store = bst.prepare_idx4_compress_store(s["keys"], s["ptr"], s["start"], None, case["rows"], ROTARY,
                                                    SECTIONS, THETA, s["ring"], None, s["table"], cache)
        return [store, bst.prepare_idx4_load(cache, s["look"], s["out"])]
    if op == "score":
        return [bst.prepare_idx4_score(s["q"], cache, s["table"], s["ptr"], s["pos"], s["max_vis"], s["scores"],
                                       s["len"])]
    cache = bst.KV8Cache(s["codes"], s["scales"])
    ws = s["workspace"] = bst.attn_workspace(DEV)
    if op == "slots":
        return [bst.prepare_attn_slots(s["q"], cache, s["slots"], s["out"], count=s["count"], lse=s["lse"],
                                       workspace=ws)]
    return [bst.prepare_attn_window(s["q"], cache, s["table"], s["ptr"], s["pos"], case["rows"], case["window"],
                                    case["sinks"], s["out"], lse=s["lse"], workspace=ws)]


def _own_outputs(s):
    op = s["case"]["op"]
    if op == "pages":
        return _page_outputs(s["ptr"], s["pos"], s["slots"], s["table"], s["ring"], s["mid"], s["end"])
    if op == "kv8":
        return s["k_out"], s["v_out"]
    if op == "keys":
        return (s["out"], s["ring"]) if s["case"]["c"] == 4 else s["out"]
    return (s["scores"], s["len"]) if op == "score" else (s["out"], s["lse"])


# ---------------------------------------------------------------- plain forms

def _power(e):
    """2^e, exactly, for whole e in -126 .. 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _page_outputs(ptr, pos, slots, table, ring, mid, end):
    return dict(ptr=ptr, pos=pos, slots=slots, table=table, ring=ring, len=mid[0], held=mid[1], pool=mid[2],
                len_end=end[0], held_end=end[1], pool_end=end[2])


def _plain_pages(s):
    table, ring, rows = s["table"].long(), s["ring"].long(), s["pos"].shape[0]
    n_req, stride = table.shape
    size, zero = ring.shape[0], s["kv_len"].new_zeros(1)
    length, held = s["kv_len"].long(), s["held"].long()
    head, count = s["pool"][0].long(), s["pool"][1].long()
    i = torch.arange(stride, device=DEV)
    # pages for the new tokens, in the order of the requests
    n = torch.minimum(s["new_len"].long().clamp(min=0), stride * PAGE - length)
    before = torch.cumsum(n, 0) - n
    n = torch.minimum(n, (rows - before).clamp(min=0))
    last = torch.cumsum(n, 0)
    want = ((length + n + PAGE - 1) // PAGE - held).clamp(min=0)
    first = torch.cumsum(want, 0) - want
    got = torch.minimum(want, (count - first).clamp(min=0))
    fresh = (i >= held[:, None]) & (i < (held + got)[:, None])
    table = torch.where(fresh, ring[(head + first[:, None] + i - held[:, None]) % size], table)
    taken = torch.minimum(want.sum(), count)
    mid = (length + n, held + got, torch.stack([(head + taken) % size, count - taken, want.sum() - taken,
                                                torch.zeros_like(taken)]))
    # rows
    r = torch.arange(rows, device=DEV)
    req = torch.searchsorted(last, r, right=True).clamp(max=n_req - 1)
    pos = torch.where(r < last[-1], length[req] + r - (last - n)[req], -1)
    page = table[req, pos.clamp(min=0) // PAGE]
    slots = torch.where((pos >= 0) & (page >= 0), page * PAGE + pos % PAGE, -1)
    # pages given back
    length, held = mid[0], mid[1]
    keep = torch.where(s["keep_len"].long() < 0, length, torch.minimum(s["keep_len"].long(), length))
    left = torch.minimum(held, (keep + PAGE - 1) // PAGE)
    gone = (i >= left[:, None]) & (i < held[:, None])
    head, count = mid[2][0], mid[2][1]
    order = torch.cumsum(gone.flatten().long(), 0).view_as(gone) - 1
    at = torch.where(gone, (head + count + order) % size, size)
    ring = torch.cat([ring, ring[:1]]).scatter(0, at.flatten(), table.flatten())[:size]
    table = torch.where(gone, -1, table)
    end = (keep, left, torch.stack([head, count + gone.sum(), torch.zeros_like(head), torch.zeros_like(head)]))
    return _page_outputs(torch.cat([zero, last.int()]), pos.int(), slots.int(), table.int(), ring.int(),
                         [x.int() for x in mid], [x.int() for x in end])


def _exponent8(top):
    """The least e with top <= 448 * 2^e, within the exponents of a scale."""
    mantissa, e = torch.frexp(top)                        # top = mantissa * 2^e, mantissa in [1/2, 1)
    e = e - 9 + (mantissa > 0.875).int()
    return torch.where(top > 0, e.clamp(KV8_EMIN, KV8_EMAX), KV8_EMIN)


def _codes8(x):
    """E4M3 codes of x (scaled), nearest, ties to even, at most 448; NaN for what is not finite."""
    y = torch.where(torch.isfinite(x), x.clamp(-KV8_TOP, KV8_TOP), math.nan)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _values8(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale


def _pool8(k, v):
    """K and V of whole pages [pages * 64, hkv, D] -> codes [pages * 64, hkv, 2, D], scales [pages, hkv, 2]."""
    x = torch.stack([k, v], 2)
    top = x.abs().amax(-1).unflatten(0, (-1, PAGE)).amax(1)
    e = _exponent8(top)
    return _codes8(x * _power(-e).repeat_interleave(PAGE, 0)[..., None]), _power(e)


def _plain_kv8(s):
    slots, pages = s["slots"].long(), s["scales"].shape[0]
    x = torch.stack([s["k"].float(), s["v"].float()], 2)                  # T, hkv, 2, D
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    page = torch.where(slots >= 0, slots // PAGE, pages)                  # padding goes to a page of its own
    most = torch.zeros((pages + 1, *top.shape[1:]), device=DEV)
    most = most.scatter_reduce(0, page[:, None, None].expand_as(top), top, "amax")[:pages]
    begun = torch.zeros(pages + 1, dtype=torch.bool, device=DEV)
    begun[torch.where(slots % PAGE == 0, page, pages)] = True
    was = torch.frexp(s["scales"]).exponent - 1
    e = _exponent8(most)
    e = torch.where(begun[:pages, None, None], e, torch.maximum(e, was))
    codes = s["codes"].unflatten(0, (pages, PAGE))
    codes = torch.where((e > was)[:, None, :, :, None],
                        _codes8(_values8(codes, _power(was - e)[:, None, :, :, None])), codes).flatten(0, 1)
    mine = _codes8(x * _power(-torch.cat([e, e[:1]]))[page][..., None])
    # rows without a slot are written behind the pool and cut off
    codes = torch.cat([codes, codes[:1]]).index_copy(0, torch.where(slots >= 0, slots, pages * PAGE), mine)[:pages * PAGE]
    at = s["look"].long()
    y = _values8(codes[at], _power(e)[at // PAGE][..., None]).to(s["k"].dtype)
    return y[:, :, 0].contiguous(), y[:, :, 1].contiguous()


def _quantise4(x):
    """x [..., D] -> E2M1 codes [..., D/2], scale bytes [..., D/32], both uint8."""
    x = x.float().unflatten(-1, (-1, GROUP))
    top = x.abs().amax(-1)
    e = (torch.frexp(top).exponent - 3).clamp(FP4_EMIN, FP4_EMAX)
    e = torch.where(top > 0, e, FP4_EMIN)
    y = x * _power(-e)[..., None]
    m = y.abs()
    # nearest of 0, .5, 1, 1.5, 2, 3, 4, 6; a value halfway goes to the even code
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _values4(codes, scales):
    """codes [..., D/2], scale bytes [..., D/32] -> the 32-bit values they stand for, [..., D]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    m = (c & 7).float()
    mag = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2.0, 2.0 * m - 8.0))
    mag = torch.where(c >= 8, -mag, mag).unflatten(-1, (-1, GROUP))
    return (mag * _power(scales.int() - 127)[..., None]).flatten(-2)


def _compressed(s):
    """The c = 4 keys of the blocks that the call completes, in 64 bits (the angles of far positions need them; the mean
    is of 32-bit sums in order), rounded to bf16."""
    b, j = s["blocks"][:, 0], s["blocks"][:, 1]
    p = 4 * j[:, None] + torch.arange(4, device=DEV)
    start = s["start"].long()[b][:, None]
    row = (s["ptr"].long()[b][:, None] + p - start).clamp(0, s["keys"].shape[0] - 1)
    raw = torch.where((p >= start)[..., None], s["keys"][row].float(), s["ring"][b].float())
    mean = ((((raw[:, 0] + raw[:, 1]) + raw[:, 2]) + raw[:, 3]) * 0.25).double()
    y = mean / mean.square().sum(-1, keepdim=True).sqrt()
    angle = (4 * j.double())[:, None] * THETA ** (-2.0 * torch.arange(ROTARY // 2, device=DEV).double() / ROTARY)
    cos, sin = torch.cos(angle), torch.sin(angle)
    lo, hi = y[:, :ROTARY // 2], y[:, ROTARY // 2:]
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], 1).to(torch.bfloat16)


def _plain_keys(s):
    if s["case"]["c"] == 4:
        # slot u of the ring: the newest token at a position of 4 i + u, if it is new
        start, n = s["start"].long()[:, None], s["case"]["rows"]
        end = start + n - 1
        p = end - (end - torch.arange(4, device=DEV)) % 4
        row = (s["ptr"].long()[:-1, None] + p - start).clamp(min=0)
        return _values4(*_quantise4(_compressed(s))), torch.where((p >= start)[..., None], s["keys"][row], s["ring"])
    return torch.where((s["slots"] >= 0)[:, None], _values4(*_quantise4(s["keys"])), 0.0)


def _padded_rows(s):
    """row [B, R]: each request's rows, its first in the place of those that it has not; valid [B, R]."""
    ptr = s["ptr"].long()
    start, n = ptr[:-1], ptr[1:] - ptr[:-1]
    i = torch.arange(s["case"]["rows"], device=DEV)
    return torch.where(i < n[:, None], start[:, None] + i, start[:, None]), i < n[:, None]


def _plain_score(s):
    c, vis = s["case"]["c"], s["max_vis"]
    j = torch.arange(vis, device=DEV)
    page = s["table"].long()[:, j * c // PAGE].clamp(min=0)
    k = _values4(*(x[page * (PAGE // c) + j % (PAGE // c)] for x in (s["codes"], s["scales"])))     # B, N, 128
    row, valid = _padded_rows(s)
    q = _values4(*_quantise4(s["q"]))[row].flatten(1, 2)                                           # B, R*4, 128
    x = torch.matmul(q, k.transpose(1, 2).contiguous()).clamp_(min=0.0)
    x = x.unflatten(1, (-1, IDX_HEADS)).sum(2) * (1.0 / math.sqrt(IDX_DIM))
    n = ((s["pos"] + 1) // c).clamp(max=vis)
    out = s["scores"].clone()
    out[:, :vis] = torch.where(j < n[:, None], x[valid], out[:, :vis])
    return out, n.int()


def _rows_at(s, slots):
    """K and V of the slots (any shape; below 0: zeros) in 32 bits, [..., hkv, D] each."""
    at = slots.long().clamp(min=0)
    kv = torch.where((slots >= 0)[..., None, None, None], _values8(s["codes"][at], s["scales"][at // PAGE][..., None]), 0.0)
    return kv[..., 0, :], kv[..., 1, :]


def _attend(q, k, v, seen):
    """q [B, R, hq, D], k and v [B, N, hkv, D], seen [B, R, N] -> out [B, R, hq, D], lse [B, R, hq]."""
    b, r, hq, d = q.shape
    hkv = k.shape[2]
    q = q.float().unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)          # B, hkv, G*R, D
    x = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * (1.0 / math.sqrt(d))
    x = x.unflatten(2, (-1, r)).masked_fill_(~seen[:, None, None], -math.inf)           # B, hkv, G, R, N
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    lse = torch.log(total) + top
    out = torch.matmul(x.flatten(2, 3), v.permute(0, 2, 1, 3).contiguous()).unflatten(2, (-1, r))
    out = torch.where(total > 0, out / total, 0.0)
    lse = torch.where(total > 0, lse, -math.inf)
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3), lse[..., 0].permute(0, 3, 1, 2).flatten(2, 3)


def _plain_slots(s):
    k, v = _rows_at(s, s["slots"])
    out, lse = _attend(s["q"][:, None], k, v, (s["slots"] >= 0)[:, None])
    return out[:, 0].to(s["q"].dtype), lse[:, 0]


def _plain_window(s):
    case, pos = s["case"], s["pos"].long()
    window, sinks, most = case["window"], case["sinks"], case["rows"]
    row, valid = _padded_rows(s)
    t = pos[row]
    first = (t[:, :1] - window + 1).clamp(min=sinks)
    j = torch.arange(sinks + window + most - 1, device=DEV)
    p = torch.where(j < sinks, j, first + j - sinks)                                     # B, N
    seen = (p[:, None] <= t[..., None]) & ((p[:, None] > t[..., None] - window) | (p[:, None] < sinks))
    page = torch.gather(s["table"].long(), 1, (p // PAGE).clamp(max=s["table"].shape[1] - 1))
    slot = torch.where(p <= t.amax(1, keepdim=True), page * PAGE + p % PAGE, -1)
    k, v = _rows_at(s, slot)
    out, lse = _attend(s["q"][row], k, v, seen)
    return out[valid].to(s["q"].dtype), lse[valid]


_PLAIN = {"pages": _plain_pages, "kv8": _plain_kv8, "keys": _plain_keys, "score": _plain_score, "slots": _plain_slots,
          "window": _plain_window}


def run(state):
    if own:
        for call in state["calls"]:
            call()
        return _own_outputs(state)
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "pages":                 # lengths and pages held in and out twice, each row's position and slot, and
        ctx, new = _contexts(case), _new_counts(case)  # each new page from the ring into the table
        pages = sum(-(-(t + n) // PAGE) + -t // PAGE for t, n in zip(ctx, new))
        return {"bytes": case["req"] * 4.0 * 12 + (sum(new) + case["pad"]) * 8.0 + pages * 8.0 + 64, "flops": 0.0}
    if op == "kv8":                   # K, V in, codes out; the filled part of the touched pages, codes in, values out
        hkv, d, size = case["hkv"], case["d"], SIZES[case["type"]]
        n = case["req"] * case["rows"]
        look = n + sum(_offsets(case))
        return {"bytes": n * (4.0 + 2 * hkv * d * (size + 1)) + look * (4.0 + 2 * hkv * d * (1 + size)),
                "flops": 2.0 * hkv * d * (n + look)}
    rec = IDX_DIM / 2 + IDX_DIM / GROUP
    if op == "keys":
        c, n = case["c"], case["req"] * case["rows"]
        keys = n if c == 1 else sum((o + case["rows"]) // 4 - o // 4 for o in _offsets(case))
        return {"bytes": n * (4.0 + IDX_DIM * SIZES[case["type"]]) + keys * (2 * rec + 4 + 4 * IDX_DIM),
                "flops": 4.0 * keys * IDX_DIM}
    ctx, rows = _contexts(case), _row_counts(case)
    bytes_, flops = 0.0, 0.0
    if op == "score":
        for t, n in zip(ctx, rows):
            c = case["c"]
            pairs = n * ((t + 1 - n / 2) // c)
            bytes_ += n * (IDX_HEADS * IDX_DIM * 2 + 8) + t // c * rec + t / PAGE * 4 + pairs * 4
            flops += 2.0 * IDX_HEADS * IDX_DIM * pairs
        return {"bytes": bytes_, "flops": flops}
    hq, hkv, d, size = case["hq"], case["hkv"], case["d"], SIZES[case["type"]]
    rec = hkv * (2 * d + 8 / PAGE)
    for t, n in zip(ctx, rows):
        io = n * hq * (2 * d * size + 4)
        if op == "slots":
            c, k = case["c"], case["k"]
            vis = t // c
            take = min(k, vis)
            keys = n * (take * c + c / 2)
            distinct = min(t, vis * (1 - (1 - take / max(1, vis)) ** n) * c + c)  # rows of a request share keys
            bytes_ += io + n * 4 * (k * c + c - 1) + distinct * rec
        else:
            s, w = case["sinks"], case["window"]
            first = max(0, t - n - w + 1)
            distinct = (t - first) + min(s, first)
            keys = 0.5 * n * (min(t, w + s) + min(t - n + 1, w + s))
            bytes_ += io + distinct * rec + distinct / PAGE * 4
        flops += 4.0 * keys * hq * d
    return {"bytes": bytes_, "flops": flops}


# ---------------------------------------------------------------- 64 bits

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e4m3_table():
    """The values of codes 0 .. 126, in order."""
    return [(m / 8.0 if e == 0 else 1 + m / 8.0) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127]


def _exact_nearest(x, grid):
    """x >= 0 to the nearest entry of an increasing grid that starts at 0, halfway cases to the even index."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    up = torch.searchsorted(grid, x.contiguous()).clamp(1, grid.shape[0] - 1)
    below, above = x - grid[up - 1], grid[up] - x
    take = (above < below) | ((above == below) & (up % 2 == 0))
    return grid[torch.where(take, up, up - 1)]


def _exact_two(e):
    table = torch.tensor([2.0 ** i for i in range(-300, 301)], dtype=torch.float64, device=e.device)
    return table[e.long() + 300]


def _exact_log2(top):
    """floor(log2 top) of positive numbers."""
    e = torch.floor(torch.log2(top))
    return e + (_exact_two(e + 1) <= top).double() - (_exact_two(e) > top).double()


def _exact_round4(x):
    """What the 4-bit form keeps of x [..., D], in 64 bits."""
    x = x.double().reshape(*x.shape[:-1], -1, GROUP)
    top = x.abs().max(dim=-1, keepdim=True).values
    e = torch.where(top > 0, _exact_log2(torch.where(top > 0, top, 1.0)) - 2, float(FP4_EMIN))
    unit = _exact_two(e.clamp(FP4_EMIN, FP4_EMAX))
    return (torch.sign(x) * _exact_nearest(x.abs() / unit, _E2M1) * unit).reshape(*x.shape[:-2], -1)


def _exact_values4(codes, scales):
    grid = torch.tensor(_E2M1 + [-x for x in _E2M1], dtype=torch.float64, device=codes.device)
    c = codes.to(torch.int32)
    x = torch.empty(c.shape[:-1] + (2 * c.shape[-1],), dtype=torch.float64, device=c.device)
    x[..., 0::2], x[..., 1::2] = grid[c % 16], grid[c // 16]
    return x * _exact_two(scales.long() - 127).repeat_interleave(GROUP, dim=-1)


def _exact_values8(codes, scale):
    table = _e4m3_table() + [math.nan]
    grid = torch.tensor(table + [-x for x in table], dtype=torch.float64, device=codes.device)
    return grid[codes.long()] * scale.double()


def _exact_kv8(s):
    slots, look = s["slots"].tolist(), s["look"].long()
    out = []
    held = {}
    for t, x in enumerate(slots):
        if x >= 0:
            held.setdefault(x // PAGE, []).append(t)
    of_page = torch.full((s["scales"].shape[0],), -1, dtype=torch.int64)
    for i, p in enumerate(held):
        of_page[p] = i
    for w, x in enumerate((s["k"].double(), s["v"].double())):
        unit, old = [], []
        for p, ts in held.items():
            top = x[ts].abs().amax((0, 2))
            e = _exact_log2(top)
            e = (e - 8 + (top > 448 * _exact_two(e - 8)).double()).clamp(KV8_EMIN, KV8_EMAX)
            was = s["scales"][p, :, w].double()
            anew = any(slots[t] % PAGE == 0 for t in ts)
            unit.append(_exact_two(e) if anew else torch.maximum(_exact_two(e), was))
            old.append(was)
        unit, old = torch.stack(unit), torch.stack(old)
        at = of_page.to(look.device)[look // PAGE]
        y = _exact_values8(s["codes"][look, :, w], old[at][..., None])
        row = torch.full((s["codes"].shape[0],), -1, dtype=torch.int64)
        row[[v for v in slots if v >= 0]] = torch.tensor([t for t, v in enumerate(slots) if v >= 0])
        row = row.to(look.device)[look]
        y = torch.where((row >= 0)[:, None, None], x[row.clamp(min=0)], y)
        u = unit[at][..., None]
        out.append(torch.sign(y) * _exact_nearest((y.abs() / u).clamp(max=448.0), _e4m3_table()) * u)
    return tuple(out)


def _exact_keys(s):
    if s["case"]["c"] == 1:
        return torch.where((s["slots"] >= 0)[:, None], _exact_round4(s["keys"]), 0.0)
    keys = []
    start, ptr = s["start"].tolist(), s["ptr"].tolist()
    for b, (o, a) in enumerate(zip(start, ptr)):
        first = o // 4 * 4
        raw = torch.cat([s["ring"][b, :o - first], s["keys"][a:ptr[b + 1]]]).float()
        raw = raw[:raw.shape[0] // 4 * 4].reshape(-1, 4, IDX_DIM)
        mean = (raw[:, 0] + raw[:, 1] + raw[:, 2] + raw[:, 3]).double() / 4
        y = mean / torch.sqrt((mean * mean).sum(1, keepdim=True))
        p = first + 4 * torch.arange(y.shape[0], device=y.device, dtype=torch.float64)
        i = torch.arange(ROTARY // 2, device=y.device, dtype=torch.float64)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=y.device),
                           p[:, None] * torch.exp(i * (-2.0 / ROTARY * math.log(THETA))))
        z = torch.complex(y[:, :64], y[:, 64:]) * turn
        keys.append(torch.cat([z.real, z.imag], 1))
    return _exact_round4(torch.cat(keys).to(torch.bfloat16)), None


def _exact_score(s):
    c = s["case"]["c"]
    out, n = s["scores"].double(), ((s["pos"].long() + 1) // c).clamp(max=s["max_vis"])
    q = _exact_round4(s["q"])
    ptr = s["ptr"].tolist()
    for b in range(s["case"]["req"]):
        for r0 in range(ptr[b], ptr[b + 1], 1024):
            r1 = min(ptr[b + 1], r0 + 1024)
            most = int(n[r0:r1].max())
            j = torch.arange(most, device=q.device)
            at = s["table"][b].long()[j * c // PAGE] * (PAGE // c) + j % (PAGE // c)
            k = _exact_values4(s["codes"][at], s["scales"][at])
            x = sum(torch.relu(q[r0:r1, h] @ k.T) for h in range(IDX_HEADS)) / math.sqrt(IDX_DIM)
            out[r0:r1, :most] = torch.where(j < n[r0:r1, None], x, out[r0:r1, :most])
    return out, None


def _exact_softmax(x, v):
    """x [m, n] scores (-inf: not seen), v [n, d]: softmax(x) v and the log of the sum."""
    top = x.max(dim=1, keepdim=True).values
    w = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = w.sum(dim=1, keepdim=True)
    some = (total > 0)[:, 0]
    out = torch.zeros((x.shape[0], v.shape[1]), dtype=torch.float64, device=x.device)
    lse = torch.full((x.shape[0],), -math.inf, dtype=torch.float64, device=x.device)
    out[some] = (w[some] @ v) / total[some]
    lse[some] = top[some, 0] + torch.log(total[some, 0])
    return out, lse


def exact(case, seed):
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    if case["op"] in ("kv8", "keys", "score"):
        return {"kv8": _exact_kv8, "keys": _exact_keys, "score": _exact_score}[case["op"]](s)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    q = s["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    heads = [slice(h * hq // hkv, (h + 1) * hq // hkv) for h in range(hkv)]

    def rows_of(slots):
        x = _exact_values8(s["codes"][slots], s["scales"][slots // PAGE][..., None])
        return x[:, :, 0], x[:, :, 1]

    if case["op"] == "slots":
        for r in range(q.shape[0]):
            k, v = rows_of(s["slots"][r][s["slots"][r] >= 0].long())
            for h, at in enumerate(heads):
                if k.shape[0]:
                    out[r, at], lse[r, at] = _exact_softmax(q[r, at] @ k[:, h].T / math.sqrt(d), v[:, h])
        return out, lse
    ptr = s["ptr"].tolist()
    for b in range(case["req"]):
        r0, r1 = ptr[b], ptr[b + 1]
        t = s["pos"][r0:r1].long()
        low = max(0, int(t.min()) - case["window"] + 1)
        p = torch.arange(int(t.max()) + 1, device=DEV)
        p = p[(p < case["sinks"]) | (p >= low)]
        k, v = rows_of(s["table"][b].long()[p // PAGE] * PAGE + p % PAGE)
        hidden = (p > t[:, None]) | ((p <= t[:, None] - case["window"]) & (p >= case["sinks"]))
        for h in range(hq):
            x = q[r0:r1, h] @ k[:, h * hkv // hq].T / math.sqrt(d)
            out[r0:r1, h], lse[r0:r1, h] = _exact_softmax(x.masked_fill(hidden, -math.inf), v[:, h * hkv // hq])
    return out, lse
