"""The attention calls at the edges of their types and sizes, against the 64-bit
references of attn_ref.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scoring_top_amd as bst
from attn_ref import attend_row, check_rows
from gpu_util import say
from test_gpu_attention import _cache, _f64, _queries

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
