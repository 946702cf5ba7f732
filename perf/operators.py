"""Cases, plain forms and 64-bit values of the KV-cache and attention operators.

Four operators follow the indexer's selection.  ``kv4_store`` quantises new K/V
rows into a paged 4-bit cache and ``kv4_load`` reads rows back; ``attn_slots``
is grouped-query attention over the KV slots that the selection emitted for
each row; ``attn_window`` is causal attention over a sliding window plus the
first tokens of each request, through the page table.

4-bit form: per (slot, kv head) D/2 bytes of K codes then D/2 bytes of V codes
(E2M1, element 2i in the low nibble of byte i), and D/32 bytes of K scales then
D/32 of V scales (one biased power of two per 32 channels).

``run`` computes the plain form in elementary torch operations in 32 bits, or,
where ``own`` is true, makes the framework's calls.
"""
import math

import torch

own = False

PAGE = 64
GROUP = 32
E_MIN, E_MAX = -120, 125
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of each of 64 requests, written and read back: latency counts
        dict(name="store_decode_64", op="store", tokens=64, hkv=2, d=128, type="bf16", fused=True, pad=0),
        # a prefill chunk's K/V
        dict(name="store_prefill_8k", op="store", tokens=8192, hkv=8, d=128, type="bf16", fused=False, pad=0),
        # an odd batch with padding rows (slot -1), heads of 64, 32-bit inputs
        dict(name="store_odd_1003", op="store", tokens=1003, hkv=5, d=64, type="f32", fused=True, pad=21),
        # the slots of one decode row (512 blocks of 4 and 2 pending tokens)
        dict(name="load_row_2050", op="load", slots=2050, hkv=2, d=128, type="bf16", pad=0),
        # the slots of 64 rows gathered for a dense consumer, some of them padding
        dict(name="load_64x2051", op="load", slots=131264, hkv=4, d=128, type="f16", pad=999),
        # one decode row at 8,192 tokens + 2 pending, c = 4, top-512
        dict(name="slots_decode_1x8k", op="slots", req=1, rows=1, lo=8194, hi=8194, c=4, k=512, hq=16, hkv=2, d=128,
             type="bf16", form="kv4"),
        # 16 decode rows at 81,920 tokens, c = 1, top-2048
        dict(name="slots_16x80k", op="slots", req=16, rows=1, lo=81920, hi=81920, c=1, k=2048, hq=32, hkv=4, d=128,
             type="bf16", form="kv4"),
        # speculative verify: 64 requests of 4K to 131K tokens, 6 rows each, c = 4, top-512
        dict(name="slots_verify_64x6", op="slots", req=64, rows=6, lo=4096, hi=131072, c=4, k=512, hq=16, hkv=2,
             d=128, type="bf16", form="kv4"),
        # rows of a prefill chunk over the 16-bit pool, heads of 64, fp16
        dict(name="slots_prefill_kv16", op="slots", req=1, rows=777, lo=32768, hi=32768, c=4, k=512, hq=24, hkv=3,
             d=64, type="f16", form="kv16"),
        # decode over a window of 4,096 and 4 first tokens, 64 requests, 4-bit cache
        dict(name="window_decode_64", op="window", req=64, rows=1, lo=4096, hi=131072, window=4096, sinks=4, hq=16,
             hkv=2, d=128, type="bf16", form="kv4"),
        # an odd ragged batch: 5 requests of 301 to 1,505 rows, odd window, 4-bit cache
        dict(name="window_ragged_5", op="window", req=5, rows=1505, lo=1600, hi=20001, window=1021, sinks=13, hq=12,
             hkv=4, d=128, type="f16", form="kv4"),
        # an 8,192-row prefill chunk of a 64K context, 16-bit pool
        dict(name="window_prefill_8k", op="window", req=1, rows=8192, lo=65536, hi=65536, window=4096, sinks=4, hq=16,
             hkv=2, d=128, type="bf16", form="kv16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "load", "slots", "window"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    kind = rng.choice(["bf16", "bf16", "f16"])
    if op == "store":
        tokens = _log(rng, 1, 8192)
        return dict(op=op, tokens=tokens, hkv=hkv, d=min(d, 1024 // hkv), type=rng.choice(["bf16", "f16", "f32"]),
                    fused=rng.random() < 0.5, pad=rng.randint(0, max(0, tokens // 50)))
    if op == "load":
        slots = _log(rng, 1, 131264 * 4 * 128 // (max(hkv, 4) * max(d, 128)))
        return dict(op=op, slots=slots, hkv=hkv, d=d, type=rng.choice(["bf16", "f16"]),
                    pad=rng.randint(0, max(0, slots // 50)))
    group = rng.choice([1, 4, 7, 8, 16])
    form = rng.choice(["kv4", "kv4", "kv16"])
    if op == "slots":
        c = rng.choice([1, 4])
        k = _log(rng, 16, 512) if c == 4 else _log(rng, 64, 2048)
        hi = _log(rng, 600, 100000)
        lo = max(64, int(hi * rng.uniform(0.1, 1)))
        rows = rng.choice([1, 1, 1, 2, 6, _log(rng, 32, 512)])
        req = 1 if rows > 6 else _log(rng, 1, 48)
        # at most what the verify case reads: 384 rows x 2,051 slots x 2 heads of 128
        while req * rows * c * k * hkv * d > 384 * 2051 * 2 * 128 and max(req, rows) > 1:
            req, rows = (req // 2, rows) if req > 1 else (req, rows // 2)
        while req * hi * hkv * d > 16 * 81920 * 4 * 128 and req > 1:  # the pool of the 80K case
            req //= 2
        return dict(op=op, req=req, rows=min(rows, lo), lo=lo, hi=hi, c=c, k=k, hq=hkv * min(group, 8), hkv=hkv, d=d,
                    type=kind, form=form)
    hi = _log(rng, 300, 60000)
    lo = max(64, int(hi * rng.uniform(0.1, 1)))
    window, sinks = _log(rng, 16, 4096), rng.choice([0, 1, 4, rng.randint(5, 100)])
    rows = rng.choice([1, 1, 6, _log(rng, 50, 2000)])
    req = _log(rng, 1, 48) if rows <= 6 else rng.randint(1, 3)
    hkv = min(hkv, 4)
    while req * hi * hkv * d > 16 * 81920 * 4 * 128 and req > 1:
        req //= 2
    while req * rows * (window + rows) * hkv * min(group, 8) * d > 8192 * 8192 * 16 * 128 // 2 and rows > 1:
        rows //= 2
    return dict(op=op, req=req, rows=min(rows, lo), lo=lo, hi=hi, window=window, sinks=sinks, hq=hkv * min(group, 8),
                hkv=hkv, d=d, type=kind, form=form)


def _contexts(case):
    """Tokens of each request, spread evenly over the logarithm of lo .. hi."""
    n, lo, hi = case["req"], case["lo"], case["hi"]
    return [int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]


def _row_counts(case):
    """Query rows of each request: all alike, or (prefill of several requests) growing to `rows`."""
    n, rows = case["req"], case["rows"]
    return [rows if rows <= 6 else max(1, rows * (i + 1) // n) for i in range(n)]


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


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
    return table, torch.tensor(ptr, dtype=torch.int32, device=DEV), torch.cat(pos), sum(pages)


def _pools(case, g, pages):
    """The cache: (codes, scales) or (K pool, V pool)."""
    hkv, d = case["hkv"], case["d"]
    k, v = (_rows(g, pages * PAGE, hkv, d) for _ in range(2))
    if case["form"] == "kv16":
        return k.to(TYPES[case["type"]]), v.to(TYPES[case["type"]])
    (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
    return torch.stack([kc, vc], 2), torch.stack([ks, vs], 2)


def prepare(case, seed):
    g = _gen(seed)
    hkv, d, kind = case["hkv"], case["d"], TYPES[case["type"]]
    s = dict(case=case)
    if case["op"] in ("store", "load"):
        n = case["tokens"] if case["op"] == "store" else case["slots"]
        pages = -(-n // PAGE) + 16
        slots = torch.randperm(pages * PAGE, generator=g, device=DEV, dtype=torch.int32)[:n].contiguous()
        if case["pad"]:
            slots[torch.randperm(n, generator=g, device=DEV)[:case["pad"]]] = -1
        s["slots"] = slots
        if case["op"] == "store":
            if case["fused"]:  # K and V as they lie in the output of a fused q/k/v projection
                qkv = torch.cat([_rows(g, n, 2 * hkv, d), _rows(g, n, 2 * hkv, d)], 1).to(kind)
                s["k"], s["v"] = qkv[:, 2 * hkv:3 * hkv], qkv[:, 3 * hkv:]
            else:
                s["k"], s["v"] = (_rows(g, n, hkv, d).to(kind) for _ in range(2))
            s["codes"] = torch.zeros((pages * PAGE, hkv, 2, d // 2), dtype=torch.uint8, device=DEV)
            s["scales"] = torch.zeros((pages * PAGE, hkv, 2, d // GROUP), dtype=torch.uint8, device=DEV)
        else:
            s["codes"], s["scales"] = _pools(dict(case, form="kv4"), g, pages)
        s["k_out"], s["v_out"] = (torch.empty((n, hkv, d), dtype=kind, device=DEV) for _ in range(2))
    else:
        s["table"], s["ptr"], s["pos"], pages = _layout(case, g)
        s["pool"] = _pools(case, g, pages)
        rows, hq = s["pos"].shape[0], case["hq"]
        s["q"] = (1.2 * torch.randn((rows, hq, d), generator=g, device=DEV)).to(kind)
        s["out"] = torch.empty((rows, hq, d), dtype=kind, device=DEV)
        s["lse"] = torch.empty((rows, hq), dtype=torch.float32, device=DEV)
        if case["op"] == "slots":
            s["slots"], s["count"] = _selection(case, s, g)
    if own:
        s["calls"] = _own_calls(s)
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


# ---------------------------------------------------------------- the framework's calls

def _own_calls(s):
    """The framework's calls with their arguments marshalled once, as a serving loop over fixed buffers keeps them."""
    import block_scoring_top_amd as bst

    case = s["case"]
    if case["op"] in ("store", "load"):
        cache = bst.KV4Cache(s["codes"], s["scales"])
        calls = [bst.prepare_kv4_store(s["k"], s["v"], s["slots"], cache)] if case["op"] == "store" else []
        return calls + [bst.prepare_kv4_load(cache, s["slots"], s["k_out"], s["v_out"])]
    cache = (bst.KV4Cache if case["form"] == "kv4" else bst.KV16Cache)(*s["pool"])
    ws = s["workspace"] = bst.attn_workspace(DEV)  # a prepared call holds addresses: the state keeps the tensor
    if case["op"] == "slots":
        return [bst.prepare_attn_slots(s["q"], cache, s["slots"], s["out"], count=s["count"], lse=s["lse"],
                                       workspace=ws)]
    return [bst.prepare_attn_window(s["q"], cache, s["table"], s["ptr"], s["pos"], case["rows"], case["window"],
                                    case["sinks"], s["out"], lse=s["lse"], workspace=ws)]


# ---------------------------------------------------------------- plain forms

def _power(e):
    """2^e, exactly, for whole e in -126 .. 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """x [..., D] -> codes [..., D/2], scale bytes [..., D/32], both uint8."""
    x = x.float().unflatten(-1, (-1, GROUP))
    top = x.abs().amax(-1)
    e = (torch.frexp(top).exponent - 3).clamp(E_MIN, E_MAX)
    e = torch.where(top > 0, e, E_MIN)
    y = x * _power(-e)[..., None]
    m = y.abs()
    # nearest of 0, .5, 1, 1.5, 2, 3, 4, 6; a value halfway goes to the even code
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """codes [..., D/2], scale bytes [..., D/32] -> the 32-bit values they stand for, [..., D]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    m = (c & 7).float()
    mag = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2.0, 2.0 * m - 8.0))
    mag = torch.where(c >= 8, -mag, mag).unflatten(-1, (-1, GROUP))
    return (mag * _power(scales.int() - 127)[..., None]).flatten(-2)


def _rows_at(s, slots):
    """K and V of the slots (any shape; below 0: zeros) in 32 bits, [..., hkv, D] each."""
    at = slots.long().clamp(min=0)
    there = (slots >= 0)[..., None, None]
    if "codes" in s or s["case"]["form"] == "kv4":
        codes, scales = (s["codes"], s["scales"]) if "codes" in s else s["pool"]
        kv = _values(codes[at], scales[at])
        k, v = kv[..., 0, :], kv[..., 1, :]
    else:
        k, v = (p[at].float() for p in s["pool"])
    return torch.where(there, k, 0.0), torch.where(there, v, 0.0)


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


def _plain_store(s):
    there = s["slots"] >= 0
    at = s["slots"][there].long()
    for i, x in enumerate((s["k"], s["v"])):
        codes, scales = _quantise(x[there])
        s["codes"][at, :, i] = codes
        s["scales"][at, :, i] = scales
    return _plain_load(s)


def _plain_load(s):
    k, v = _rows_at(s, s["slots"])
    kind = TYPES[s["case"]["type"]]
    return k.to(kind), v.to(kind)


def _plain_slots(s):
    k, v = _rows_at(s, s["slots"])
    out, lse = _attend(s["q"][:, None], k, v, (s["slots"] >= 0)[:, None])
    return out[:, 0].to(s["q"].dtype), lse[:, 0]


def _plain_window(s):
    case, ptr, pos = s["case"], s["ptr"].long(), s["pos"].long()
    window, sinks, most = case["window"], case["sinks"], case["rows"]
    start, n = ptr[:-1], ptr[1:] - ptr[:-1]
    i = torch.arange(most, device=DEV)
    row = torch.where(i < n[:, None], start[:, None] + i, start[:, None])                # B, R
    t = pos[row]
    first = (t[:, :1] - window + 1).clamp(min=sinks)
    j = torch.arange(sinks + window + most - 1, device=DEV)
    p = torch.where(j < sinks, j, first + j - sinks)                                     # B, N
    seen = (p[:, None] <= t[..., None]) & ((p[:, None] > t[..., None] - window) | (p[:, None] < sinks))
    page = torch.gather(s["table"].long(), 1, (p // PAGE).clamp(max=s["table"].shape[1] - 1))
    slot = torch.where(p <= t.amax(1, keepdim=True), page * PAGE + p % PAGE, -1)
    k, v = _rows_at(s, slot)
    out, lse = _attend(s["q"][row], k, v, seen)
    valid = i < n[:, None]
    return out[valid].to(s["q"].dtype), lse[valid]


def run(state):
    op = state["case"]["op"]
    if own:
        for call in state["calls"]:
            call()
        return (state["k_out"], state["v_out"]) if op in ("store", "load") else (state["out"], state["lse"])
    return {"store": _plain_store, "load": _plain_load, "slots": _plain_slots, "window": _plain_window}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    hkv, d = case["hkv"], case["d"]
    rec4 = hkv * (d + d // 16)                       # 4-bit K and V of one slot
    size = {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
    if case["op"] == "store":                        # K, V in; codes and scales, and their values, out
        n = case["tokens"] - case["pad"]
        return {"bytes": case["tokens"] * (4 + 2 * hkv * d * size) + n * (rec4 + 2 * hkv * d * size), "flops": 4.0 * n * hkv * d}
    if case["op"] == "load":
        n = case["slots"] - case["pad"]
        return {"bytes": case["slots"] * (4 + 2 * hkv * d * size) + n * rec4, "flops": 2.0 * n * hkv * d}
    rec = rec4 if case["form"] == "kv4" else 2 * hkv * d * size
    hq, ctx, rows = case["hq"], _contexts(case), _row_counts(case)
    bytes_, flops = 0.0, 0.0
    for t, n in zip(ctx, rows):
        io = n * hq * (2 * d * size + 4)
        if case["op"] == "slots":
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


def _exact_power(e):
    """2^e in 64 bits from a table, so that values halfway between two codes stay halfway."""
    table = torch.tensor([2.0 ** i for i in range(-200, 201)], dtype=torch.float64, device=e.device)
    return table[e.long() + 200]


def _exact_round(x):
    """What the 4-bit form keeps of x [..., D], in 64 bits."""
    x = x.double().reshape(*x.shape[:-1], -1, GROUP)
    top = x.abs().max(dim=-1, keepdim=True).values
    e = torch.where(top > 0, torch.floor(torch.log2(top)), float(E_MIN))
    e = e + (_exact_power(e + 1) <= top).double() - ((_exact_power(e) > top) & (top > 0)).double()  # log2's rounding
    unit = _exact_power((e - 2).clamp(E_MIN, E_MAX))
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    best = torch.zeros_like(x)
    gap = (x.abs() / unit - 0.0).abs()
    for i in range(1, 8):
        g = (x.abs() / unit - grid[i]).abs()
        take = (g < gap) | ((g == gap) & (i % 2 == 0))
        best, gap = torch.where(take, grid[i], best), torch.where(take, g, gap)
    return (torch.sign(x) * best * unit).reshape(*x.shape[:-2], -1)


def _exact_rows(s, slots):
    """64-bit K and V of a list of slots >= 0, [n, hkv, D] each."""
    at = slots.long()
    if "codes" not in s and s["case"]["form"] == "kv16":
        return s["pool"][0][at].double(), s["pool"][1][at].double()
    codes, scales = (s["codes"], s["scales"]) if "codes" in s else s["pool"]
    grid = torch.tensor(_E2M1 + [-x for x in _E2M1], dtype=torch.float64, device=codes.device)
    c = codes[at].to(torch.int32)
    x = torch.empty(c.shape[:-1] + (2 * c.shape[-1],), dtype=torch.float64, device=c.device)
    x[..., 0::2], x[..., 1::2] = grid[c % 16], grid[c // 16]
    x = x * _exact_power(scales[at].long() - 127).repeat_interleave(GROUP, dim=-1)
    return x[:, :, 0], x[:, :, 1]


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
    s = prepare(case, seed)
    if case["op"] in ("store", "load"):
        there = s["slots"] >= 0
        if case["op"] == "store":
            got = [_exact_round(s[n]) for n in "kv"]
            return tuple(torch.where(there[:, None, None], x, torch.zeros_like(x)) for x in got)
        out = [torch.zeros(s["k_out"].shape, dtype=torch.float64, device=DEV) for _ in range(2)]
        for x, y in zip(out, _exact_rows(s, s["slots"][there])):
            x[there] = y
        return tuple(out)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    q = s["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    heads = [slice(h * hq // hkv, (h + 1) * hq // hkv) for h in range(hkv)]
    if case["op"] == "slots":
        for r in range(q.shape[0]):
            k, v = _exact_rows(s, s["slots"][r][s["slots"][r] >= 0])
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
        k, v = _exact_rows(s, s["table"][b].long()[p // PAGE] * PAGE + p % PAGE)
        hidden = (p > t[:, None]) | ((p <= t[:, None] - case["window"]) & (p >= case["sinks"]))
        for h in range(hq):
            x = q[r0:r1, h] @ k[:, h * hkv // hq].T / math.sqrt(d)
            out[r0:r1, h], lse[r0:r1, h] = _exact_softmax(x.masked_fill(hidden, -math.inf), v[:, h * hkv // hq])
    return out, lse
