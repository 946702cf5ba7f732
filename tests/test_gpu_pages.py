"""pages_extend and pages_release on the GPU against plain loops over the same
state (more_ref.py): every output exact."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scoring_top_amd as bst
from block_scoring_top_amd.pipeline import PagedBatch
from gpu_util import say
from more_ref import pages_extend, pages_release

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


class State:
    """A batch's state on both sides; each call is compared in full."""

    def __init__(self, kv_len, table, ring, pool, held=None):
        self.kv_len = list(kv_len)
        self.held = [-(-t // 64) for t in kv_len] if held is None else list(held)
        self.table, self.ring, self.pool = np.asarray(table, np.int32), np.asarray(ring, np.int32), list(pool)
        self.g = dict(kv_len=_i32(self.kv_len), held=_i32(self.held), table=_i32(self.table), pool=bst.PagePool(
            _i32(self.ring), _i32(self.pool)))

    def check(self, want, got):
        for name, x in want.items():
            y = self.g["pool"].ring if name == "ring" else got[name]
            np.testing.assert_array_equal(y.cpu().numpy(), np.asarray(x, np.int32), err_msg=name)

    def extend(self, new_len, num_rows, in_place=True):
        want = pages_extend(self.kv_len, self.held, new_len, self.table, self.ring, self.pool, num_rows)
        B = len(self.kv_len)
        g = self.g
        out = dict(ptr=torch.full((B + 1,), -9, dtype=torch.int32, device="cuda"),
                   tok_start=torch.full((B,), -9, dtype=torch.int32, device="cuda"),
                   pos=torch.full((num_rows + 1,), -9, dtype=torch.int32, device="cuda"),
                   slots=torch.full((num_rows + 1,), -9, dtype=torch.int32, device="cuda"))
        kw = {} if in_place else dict(kv_len_out=torch.empty_like(g["kv_len"]), held_out=torch.empty_like(g["held"]),
                                      pool_out=bst.PagePool(g["pool"].ring, torch.zeros(4, dtype=torch.int32, device="cuda")))
        bst.pages_extend(g["pool"], g["kv_len"], g["held"], _i32(new_len), g["table"], out["ptr"], out["pos"][:num_rows],
                         out["slots"][:num_rows], tok_start=out["tok_start"], **kw)
        torch.cuda.synchronize()
        assert out["pos"][num_rows] == -9 and out["slots"][num_rows] == -9
        if not in_place:
            assert g["kv_len"].tolist() == self.kv_len and g["pool"].state.tolist() == self.pool
            g["kv_len"], g["held"], g["pool"] = kw["kv_len_out"], kw["held_out"], kw["pool_out"]
        out["pos"], out["slots"] = out["pos"][:num_rows], out["slots"][:num_rows]
        self.check(want, dict(out, kv_len=g["kv_len"], held=g["held"], table=g["table"], pool=g["pool"].state))
        self.kv_len, self.held, self.table, self.pool = want["kv_len"], want["held"], want["table"], want["pool"]
        return want

    def release(self, keep_len, in_place=True):
        want = pages_release(self.kv_len, self.held, keep_len, self.table, self.ring, self.pool)
        g = self.g
        kw = {} if in_place else dict(kv_len_out=torch.empty_like(g["kv_len"]), held_out=torch.empty_like(g["held"]),
                                      pool_out=bst.PagePool(g["pool"].ring, torch.zeros(4, dtype=torch.int32, device="cuda")))
        bst.pages_release(g["pool"], g["kv_len"], g["held"], _i32(keep_len), g["table"], **kw)
        torch.cuda.synchronize()
        if not in_place:
            g["kv_len"], g["held"], g["pool"] = kw["kv_len_out"], kw["held_out"], kw["pool_out"]
        self.check(want, dict(kv_len=g["kv_len"], held=g["held"], table=g["table"], pool=g["pool"].state))
        self.kv_len, self.held, self.table, self.ring, self.pool = (want[n] for n in ("kv_len", "held", "table", "ring", "pool"))


def _fresh(num_req, stride, num_pages, seed=0, head=0):
    ring = np.random.default_rng(seed).permutation(num_pages)
    return State([0] * num_req, np.full((num_req, stride), -1), np.roll(ring, head), [head % num_pages, num_pages, 0, 0])


@pytest.mark.parametrize("num_req,most,steps", [(1, 200, 6), (7, 90, 8), (64, 6, 12), (300, 40, 4), (1500, 3, 4), (5000, 2, 3)])
@pytest.mark.parametrize("in_place", [True, False])
def test_random_steps(num_req, most, steps, in_place):
    """Extended, cut back, finished and extended again; the ring wraps."""
    say(f"pages random steps num_req={num_req} most={most} in_place={in_place}")
    rng = np.random.default_rng(num_req)
    s = _fresh(num_req, 1 + steps * most // 64 + 1, num_req * (2 + steps * most // 64), num_req, head=num_req // 2)
    for i in range(steps):
        new = rng.integers(0, most + 1, num_req)
        new[rng.random(num_req) < 0.1] = -3
        s.extend(new, int(np.maximum(new, 0).sum()) + int(rng.integers(0, 100)), in_place)
        keep = np.where(rng.random(num_req) < 0.2, 0, np.where(rng.random(num_req) < 0.5, -1, rng.integers(0, steps * most, num_req)))
        s.release(keep, in_place)


@pytest.mark.parametrize("rows", [4095, 4096, 4097, 8192, 40000])
def test_prompts(rows):
    """Enough rows for several workgroups, one prompt and decoding requests beside it, in place."""
    say(f"pages prompts rows={rows}")
    s = _fresh(9, 2 + rows // 64, 20 + rows // 64, 3)
    s.extend([5, 64, 0, 1, 63, 65, 7, 128, 2], 335)
    s.extend([1, 1, 0, 1, rows - 6, 1, 1, 0, 1], rows)
    s.release([-1, 3, 0, 0, rows // 2, 0, 500, 127, 64])
    s.extend([1] * 9, 4096 * 3 + 5)


def test_the_ring_runs_out():
    say("pages short")
    s = _fresh(5, 8, 4, 1, head=3)
    w = s.extend([100, 1, 70, 64, 1], 300)                     # 2 + 1 + 2: one lacking of the third, two more behind
    assert w["pool"][1:3] == [0, 3] and w["slots"].count(-1) == 300 - 165
    s.extend([0, 0, 0, 0, 0], 0)                               # still lacking
    s.release([0, -1, -1, -1, -1])
    s.extend([0, 1, 0, 0, 0], 1)                               # takes what it lacked
    s.release([0] * 5)
    assert s.pool[1] == 4


def test_limits_of_rows_and_table():
    """Tokens past the rows or the table's end are not taken; pages held from before a cut are used again."""
    say("pages limits")
    s = _fresh(4, 2, 40, 2)
    s.extend([200, 50, 100, 30], 500)                          # 200 > 128
    assert s.kv_len == [128, 50, 100, 30]
    s.extend([5, 20, 100, 3], 10)                              # rows end inside the second request
    assert s.kv_len == [128, 60, 100, 30]
    s.kv_len[2] = 10                                           # set back by the caller: 2 pages held for 10 tokens
    s.g["kv_len"][2] = 10
    s.extend([0, 0, 60, 0], 60)
    assert s.held[2] == 2 and s.pool[2] == 0
    s.release([-1] * 4)                                        # nothing to give back but unused pages
    s.kv_len[2] = 10
    s.g["kv_len"][2] = 10
    s.release([-1, -1, 1 << 30, -1])
    assert s.held[2] == 1


def test_no_requests_and_no_rows():
    say("pages empty")
    s = _fresh(3, 4, 9, 5)
    s.extend([0, 0, 0], 0)
    s.extend([-5, 0, 0], 7)
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    pool = bst.PagePool(s.g["pool"].ring, _i32([2, 5, 1, 0]))
    out = bst.PagePool(pool.ring, _i32([7, 7, 7, 0]))
    ptr, pos, slots = _i32([-9]), _i32([-9] * 3), _i32([-9] * 3)
    bst.pages_extend(pool, z, z, z, torch.empty((0, 4), dtype=torch.int32, device="cuda"), ptr, pos, slots, pool_out=out)
    torch.cuda.synchronize()
    assert out.state.tolist() == [2, 5, 0, 0] and ptr.tolist() == [0] and pos.tolist() == slots.tolist() == [-1] * 3
    bst.pages_release(pool, z, z, z, torch.empty((0, 4), dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert pool.state.tolist() == [2, 5, 0, 0]


def test_bad_state_stays_inside_the_buffers():
    """Lengths, page counts, heads and page ids out of range: guards around every buffer stay as they were."""
    say("pages bad state")
    B, stride, size, rows = 6, 3, 8, 20

    def guarded(*shape):
        whole = torch.full((shape[0] + 2, *shape[1:]), -12345, dtype=torch.int32, device="cuda")
        return whole, whole[1:-1]
    bad = [0, -7, 2**31 - 1, -2**31, 5000, 191]
    for pool in ([-5, 4, 0, 0], [2**31 - 1, 2**31 - 1, 0, 0], [3, -1, 0, 0], [7, 8, 0, 0]):
        bufs = {n: guarded(*sh) for n, sh in dict(kv=(B,), held=(B,), table=(B, stride), ring=(size,), pool=(4,), ptr=(B + 1,),
                                                  pos=(rows,), slots=(rows,)).items()}
        b = {n: v for n, (_, v) in bufs.items()}
        for held in ([3, 4, -1, 2**31 - 1, 0, 3], [0] * B):
            for change in ([1, 2**31 - 1, 2**31 - 1, -2**31, 7, 3], [2**31 - 1] * B):
                b["kv"].copy_(_i32(bad)), b["held"].copy_(_i32(held)), b["pool"].copy_(_i32(pool))
                b["ring"].copy_(_i32([0, -1, 2**31 - 1, 1 << 25, 3, 4, 5, 6])), b["table"].fill_(2**30)
                p = bst.PagePool(b["ring"], b["pool"])
                bst.pages_extend(p, b["kv"], b["held"], _i32(change), b["table"], b["ptr"], b["pos"], b["slots"])
                bst.pages_release(p, b["kv"], b["held"], _i32(change), b["table"])
                torch.cuda.synchronize()
                for n, (whole, _) in bufs.items():
                    assert (whole[0] == -12345).all() and (whole[-1] == -12345).all(), n
                assert b["ptr"].diff().min() >= 0 and b["ptr"][-1] <= rows


def test_captured_steps_and_streams():
    """A step captured once and replayed with other lengths, eager work between the replays; the same on a stream."""
    say("pages captured")
    B, rows = 40, 5000
    a, e = (PagedBatch(B, 10000, 2000, rows, "cuda") for _ in range(2))
    new, keep = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), -1, dtype=torch.int32, device="cuda")

    def step(batch):
        batch.extend(new)
        batch.release(keep)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(a)                                                # no new tokens
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
    torch.cuda.synchronize()
    rng = np.random.default_rng(0)
    for i in range(6):
        new.copy_(_i32(rng.integers(0, 120, B)))
        keep.copy_(_i32(np.where(rng.random(B) < 0.3, rng.integers(0, 300, B), -1)))
        step(e)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n in ("kv_len", "held", "page_table", "req_row_ptr", "row_pos", "slots", "tok_start"):
            assert torch.equal(getattr(a, n), getattr(e, n)), (i, n)
        assert torch.equal(a.pool.state, e.pool.state) and torch.equal(a.pool.ring, e.pool.ring)
    with torch.cuda.stream(side):
        e.extend(new)
    a.extend(new, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a.slots, e.slots) and a.pool.state[3] == 0


def test_prepared_calls():
    a, e = (PagedBatch(3, 400, 30, 200, "cuda") for _ in range(2))
    new, keep = _i32([70, 1, 64]), _i32([1, 0, -1])
    calls = (bst.prepare_pages_extend(a.pool, a.kv_len, a.held, new, a.page_table, a.req_row_ptr, a.row_pos, a.slots,
                                      tok_start=a.tok_start),
             bst.prepare_pages_release(a.pool, a.kv_len, a.held, keep, a.page_table))
    for call in (*calls, calls[0].bind()):
        call()
    e.extend(new), e.release(keep), e.extend(new)
    torch.cuda.synchronize()
    for n in ("kv_len", "held", "page_table", "req_row_ptr", "row_pos", "slots", "tok_start"):
        assert torch.equal(getattr(a, n), getattr(e, n)), n
