"""References of the page tables, the 8-bit cache and the 4-bit index scores
(numpy and plain loops, from the definitions), and the error bound of the scores.

Score bound.  Products of 4-bit values and their scales are exact; a dot product
sums 128 of them in FP32, in any order: off by at most 127 * 2^-24 of the sum of
their magnitudes to first order, 130 covers the rest.  ReLU shrinks errors; three
additions and the scaling (whose factor is itself rounded) add 5 * 2^-24 of the
result, which is no more than the sum of magnitudes: 136 * 2^-24 in all.
"""
from __future__ import annotations

import numpy as np

PAGE = 64
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)])
E4M3[127] = np.nan                                  # codes 0 .. 127; bit 7 is the sign


def e4m3_round(y):
    """Code of the value nearest to each |y| (at most 448), halfway cases to the even one; sign in bit 7; NaN: 0x7F."""
    a = np.abs(np.where(np.isfinite(y), y, 0.0))
    grid = E4M3[:127]
    up = np.clip(np.searchsorted(grid, a), 1, 126)
    below, above = a - grid[up - 1], grid[up] - a
    code = np.where((above < below) | ((above == below) & (up % 2 == 0)), up, up - 1)
    return np.where(np.isfinite(y), code + 128 * np.signbit(y), 127).astype(np.uint8)


def e4m3_value(codes):
    return np.where(codes >= 128, -1.0, 1.0) * E4M3[codes & 127]


def kv8_exponent(top):
    """The least e with top <= 448 * 2^e, clamped."""
    top = np.asarray(top, np.float64)
    _, ex = np.frexp(np.where(top > 0, top, 1.0))
    e = ex - 9                                       # 256 * 2^e <= top < 512 * 2^e
    e = np.where(top > 448.0 * np.ldexp(1.0, e), e + 1, e)
    return np.where(top > 0, np.clip(e, -120, 119), -120)


class Kv8:
    """The 8-bit cache: codes [slots, hkv, 2, D], exponents [pages, hkv, 2]."""

    def __init__(self, pages, hkv, d, codes=None, exps=None):
        self.codes = np.zeros((pages * PAGE, hkv, 2, d), np.uint8) if codes is None else codes.copy()
        self.exps = np.full((pages, hkv, 2), -120, np.int64) if exps is None else exps.copy()

    def store(self, k, v, slots):
        """k, v [T, hkv, D] float64."""
        x = np.stack([k, v], 2)
        there = (slots >= 0) & (slots < self.codes.shape[0])
        for page in np.unique(slots[there] // PAGE):
            rows = np.nonzero(there & (slots // PAGE == page))[0]
            y = x[rows]
            top = np.where(np.isfinite(y), np.abs(y), 0.0).max((0, 3))
            e = kv8_exponent(top)
            old = self.exps[page]
            if (slots[rows] % PAGE != 0).all():
                e = np.maximum(e, old)
                s = slice(page * PAGE, page * PAGE + PAGE)
                again = e4m3_round(e4m3_value(self.codes[s]) * np.ldexp(1.0, old - e)[None, :, :, None])
                again = np.where(self.codes[s] & 127 == 127, self.codes[s], again)
                self.codes[s] = np.where((e > old)[None, :, :, None], again, self.codes[s])
            self.exps[page] = e
            with np.errstate(over="ignore"):
                self.codes[slots[rows]] = e4m3_round(np.clip(y * np.ldexp(1.0, -e)[None, :, :, None], -448, 448)
                                                     if np.isfinite(y).all() else
                                                     np.where(np.isfinite(y), np.clip(np.where(np.isfinite(y), y, 0.0) * np.ldexp(
                                                         1.0, -e)[None, :, :, None], -448, 448), np.nan))

    def values(self):
        """K and V [slots, hkv, D] float64."""
        x = e4m3_value(self.codes) * np.ldexp(1.0, np.repeat(self.exps, PAGE, 0))[..., None]
        return x[:, :, 0], x[:, :, 1]


def pages_extend(kv_len, held, new_len, table, ring, pool, num_rows):
    """Plain loops over the state (lists and arrays); returns everything that the call writes, the table updated."""
    table = table.copy()
    size, stride = len(ring), table.shape[1]
    head, count = pool[0], pool[1]
    ptr, tok_start, pos, slots = [0], [], [], []
    kv_len, held = list(map(int, kv_len)), list(map(int, held))
    lacking = 0
    for b in range(len(kv_len)):
        tok_start.append(kv_len[b])
        n = max(0, min(int(new_len[b]), 64 * stride - kv_len[b], num_rows - len(pos)))
        for _ in range(max(0, -(-(kv_len[b] + n) // PAGE) - held[b])):
            if count == 0:
                lacking += 1
                continue
            table[b, held[b]] = ring[head]
            held[b] += 1
            head, count = (head + 1) % size, count - 1
        for p in range(kv_len[b], kv_len[b] + n):
            page = table[b, p // PAGE] if p // PAGE < held[b] else -1
            pos.append(p)
            slots.append(page * PAGE + p % PAGE if page >= 0 else -1)
        kv_len[b] += n
        ptr.append(len(pos))
    pad = [-1] * (num_rows - len(pos))
    return dict(kv_len=kv_len, held=held, table=table, pool=[head, count, lacking, 0], ptr=ptr, tok_start=tok_start,
                pos=pos + pad, slots=slots + pad)


def pages_release(kv_len, held, keep_len, table, ring, pool):
    table, ring = table.copy(), ring.copy()
    size = len(ring)
    head, count = pool[0], pool[1]
    kv_len, held = list(map(int, kv_len)), list(map(int, held))
    for b in range(len(kv_len)):
        if keep_len[b] >= 0:
            kv_len[b] = min(kv_len[b], int(keep_len[b]))
        for i in range(-(-kv_len[b] // PAGE), held[b]):
            ring[(head + count) % size] = table[b, i]
            count += 1
            table[b, i] = -1
        held[b] = min(held[b], -(-kv_len[b] // PAGE))
    return dict(kv_len=kv_len, held=held, table=table, ring=ring, pool=[head, count, 0, 0])


def bf16(x):
    """float64 -> bf16 by way of FP32, as float64 (finite values)."""
    u = np.asarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + (u >> 16 & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


def compressed_keys(raw, pos, rot, sections, theta):
    """raw [n, 4, 128] (bf16 values), pos [n, 3] (t, h, w of the first token): the compressed keys [n, 128] in bf16."""
    r = np.asarray(raw, np.float32)
    mean = ((((r[:, 0] + r[:, 1]) + r[:, 2]) + r[:, 3]) * np.float32(0.25)).astype(np.float64)
    norm = np.sqrt((mean * mean).sum(1, keepdims=True))
    y = np.divide(mean, norm, out=np.zeros_like(mean), where=norm > 0)
    i = np.arange(rot // 2)
    comp = np.repeat([0, 1, 2], sections)
    angle = np.asarray(pos, np.float64)[:, comp] * theta ** (-2.0 * i / max(rot, 1))
    lo, hi = y[:, :rot // 2].copy(), y[:, rot // 2:rot].copy()
    y[:, :rot // 2], y[:, rot // 2:rot] = lo * np.cos(angle) - hi * np.sin(angle), hi * np.cos(angle) + lo * np.sin(angle)
    return bf16(y)


def score_row(q, k):
    """q [4, 128], k [n, 128] float64: scores [n] and their bound."""
    x = q @ k.T
    mag = np.abs(q) @ np.abs(k).T
    return np.maximum(x, 0.0).sum(0) / np.sqrt(128.0), 136 * 2.0 ** -24 * mag.sum(0) / np.sqrt(128.0)
