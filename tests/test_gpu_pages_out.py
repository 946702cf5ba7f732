"""pages_extend and pages_release into buffers of their own that hold anything, into
some of their own and some of the state's, and into those of another argument."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scoring_top_amd as bst
from gpu_util import say
from more_ref import pages_extend, pages_release

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


@pytest.mark.parametrize("B,rows", [(3, 400), (3, 9000), (200, 30000), (700, 40000), (5000, 9000)])
@pytest.mark.parametrize("own", [("kv", "held", "pool"), ("pool",), ("kv", "held"), ("held", "pool"), ("change", "held", "pool")])
def test_outputs_of_their_own(B, rows, own):
    """``own``: which outputs are buffers of their own ("change": kv_len goes where new_len, then keep_len, was)."""
    say(f"pages outputs B={B} rows={rows} own={own}")
    rng = np.random.default_rng(B + rows)
    stride, size = rows // 64 + 8, rows // 64 + 2 * B + 5
    kv, held = np.zeros(B, int), np.zeros(B, int)
    table, ring, pool = np.full((B, stride), -1), rng.permutation(size), [size // 2, size, 0, 0]
    ring = np.roll(ring, size // 2)
    g = dict(kv=_i32(kv), held=_i32(held), pool=_i32(pool))
    gt, gr = _i32(table), _i32(ring)
    ptr, pos, slots = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (B + 1, rows, rows))

    def outs(change):
        o = {n: torch.full_like(g[n], 9 + i) if n in own else g[n] for i, n in enumerate(g)}
        if "change" in own:
            o["kv"] = change
        return o

    for i in range(4):
        new = rng.multinomial(rows - 10 * i, np.full(B, 1 / B)) if i != 1 else rng.integers(0, 3, B)
        want = pages_extend(kv, held, new, table, ring, pool, rows)
        change = _i32(new)
        o = outs(change)
        bst.pages_extend(bst.PagePool(gr, g["pool"]), g["kv"], g["held"], change, gt, ptr, pos, slots, kv_len_out=o["kv"],
                         held_out=o["held"], pool_out=bst.PagePool(gr, o["pool"]))
        g = o
        torch.cuda.synchronize()
        for name, got in dict(kv_len=g["kv"], held=g["held"], pool=g["pool"], table=gt, ptr=ptr, pos=pos, slots=slots).items():
            np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(want[name]), err_msg=f"extend {i} {name}")
        kv, held, table, pool = (want[n] for n in ("kv_len", "held", "table", "pool"))
        keep = np.where(rng.random(B) < 0.7, 0, rng.integers(-1, max(2, rows // B), B))
        want = pages_release(kv, held, keep, table, ring, pool)
        change = _i32(keep)
        o = outs(change)
        bst.pages_release(bst.PagePool(gr, g["pool"]), g["kv"], g["held"], change, gt, kv_len_out=o["kv"], held_out=o["held"],
                          pool_out=bst.PagePool(gr, o["pool"]))
        g = o
        torch.cuda.synchronize()
        for name, got in dict(kv_len=g["kv"], held=g["held"], pool=g["pool"], table=gt, ring=gr).items():
            np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(want[name]), err_msg=f"release {i} {name}")
        kv, held, table, ring, pool = (want[n] for n in ("kv_len", "held", "table", "ring", "pool"))
