"""Whole steps over the page tables, the 8-bit cache and the 4-bit index keys on
the GPU: padded batches, captured once and replayed with other lengths; calls of
two streams at once; slots named twice."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scoring_top_amd as bst
from attn_ref import attend_row, check_rows, quantise
from block_scoring_top_amd.pipeline import IndexerPath, PagedBatch
from gpu_util import say
from more_ref import Kv8, compressed_keys

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


class Step:
    """A batch with its caches and the inputs of a step, ``rows`` of them whatever the step's tokens."""

    def __init__(self, c, B, rows, cap, pages, k, hkv=2, hq=8, d=64):
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.c, self.rows, self.cap, self.pages, self.kk = c, rows, cap, pages, k
        self.batch = PagedBatch(B, cap, pages, rows, "cuda")
        self.cache, self.keys = bst.KV8Cache.empty(pages, hkv, d, "cuda"), bst.Idx4Cache.empty(pages, c, "cuda")
        self.new = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.ring = torch.zeros((B, 4, 128), **bf16)
        self.k, self.v = (torch.zeros((rows, hkv, d), **bf16) for _ in range(2))
        self.raw, self.iq = torch.zeros((rows, 128), **bf16), torch.zeros((rows, 4, 128), **bf16)
        self.q = torch.zeros((rows, hq, d), **bf16)
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros((rows, hq), dtype=torch.float32, device="cuda")
        self.path = self.scorer(rows)

    def scorer(self, rows):
        b = self.batch
        return IndexerPath(type("Inputs", (), dict(c=self.c, k=self.kk, q=self.iq[:rows], kcache=self.keys, num_pages=self.pages,
                                                   page_table=b.page_table, req_row_ptr=b.req_row_ptr, row_pos=b.row_pos[:rows],
                                                   max_vis=self.cap // self.c))(), "idx4")

    def fill(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        for x in (self.k, self.v, self.raw, self.iq, self.q):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))

    def run(self):
        b = self.batch
        b.extend(self.new)
        bst.kv8_store(self.k, self.v, b.slots, self.cache)
        if self.c == 4:
            bst.idx4_compress_store(self.raw, b.req_row_ptr, b.tok_start, None, self.rows, 64, (16, 8, 8), 10000.0, self.ring,
                                    None, b.page_table, self.keys)
        else:
            bst.idx4_store(self.raw, b.slots, self.keys)
        self.path.run()
        self.path.attend(self.q, self.cache, self.out, lse=self.lse)

    def results(self):
        b, p = self.batch, self.path
        return dict(page_table=b.page_table, kv_len=b.kv_len, slots=b.slots, pool=b.pool.state, codes=self.cache.codes,
                    scales=self.cache.scales, keys=self.keys.codes, key_scales=self.keys.scales, chosen=p.slots, sel=p.sel,
                    out=self.out, lse=self.lse)


@pytest.mark.parametrize("c,rows", [(1, 48), (4, 48), (4, 500)])
def test_padded_steps_captured(c, rows):
    """A step of `rows` rows, of which each time others are padding: captured and replayed like an eager batch, which
    agrees with the scores of the same rows without padding and with attention in 64 bits."""
    say(f"padded steps c={c} rows={rows}")
    B, cap, pages, k, d = 5, 640, 40, 64 // c, 64
    a, e = (Step(c, B, rows, cap, pages, k) for _ in range(2))
    ref, kc = Kv8(pages, 2, d), torch.zeros((pages * 64 // c, 128), dtype=torch.bfloat16, device="cuda")
    seen = {}                                                    # (request, position mod 4): raw index key
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a.run()                                                  # no tokens: nothing but padding
    torch.cuda.synchronize()
    assert (a.path.slots == -1).all() and (a.out == 0).all() and torch.isneginf(a.lse).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
    torch.cuda.synchronize()
    big = min(rows, 400)
    steps = [[big // 2, 0, 3, big // 4, 1], [1, 1, 1, 1, 1], [0] * 5, [6, 6, 1, 6, 6], [1, big - 3, 1, 0, 1], [2, 2, 0, 2, 2]]
    keep = {1: [-1, -1, 2, 7, -1], 3: [0, -1, -1, -1, 3]}
    for i, new in enumerate(steps):
        for s in (a, e):
            s.new.copy_(_i32(new))
            s.fill(i)
        e.run()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = e.results()
        for n, x in a.results().items():
            assert torch.equal(x, want[n]), (i, n)
        n = sum(new)
        ptr, table, pos = (x.cpu().numpy() for x in (e.batch.req_row_ptr, e.batch.page_table, e.batch.row_pos))
        assert ptr[-1] == n and (pos[n:] == -1).all()
        assert (e.path.slots[n:] == -1).all() and (e.out[n:] == 0).all() and torch.isneginf(e.lse[n:]).all()
        slots = e.batch.slots.cpu().numpy()
        ref.store(_f64(e.k), _f64(e.v), slots)
        if c == 4:                                               # the keys of the blocks that are whole now
            raw, starts = _f64(e.raw), e.batch.tok_start.tolist()
            for b in range(B):
                for p in range(starts[b], starts[b] + ptr[b + 1] - ptr[b]):
                    seen[b, p % 4] = raw[ptr[b] + p - starts[b]]  # a ring, which cutting back leaves as it is
                    if p % 4 == 3:
                        key = compressed_keys([[seen[b, u] for u in range(4)]], [[p - 3] * 3], 64, (16, 8, 8), 10000.0)
                        kc[int(table[b, p // 64]) * 16 + p // 4 % 16] = torch.tensor(key[0]).bfloat16()
        elif n:
            kc[e.batch.slots[:n].long()] = e.raw[:n]
        held = np.unique(table[table >= 0])
        codes, exps = quantise(_f64(kc))
        in_use = (held[:, None] * (64 // c) + np.arange(64 // c)).reshape(-1)
        written = in_use[(codes[in_use] != 0).any(1)]            # not the rest of the last pages
        np.testing.assert_array_equal(e.keys.codes.cpu().numpy()[written], codes[written])
        np.testing.assert_array_equal(e.keys.scales.cpu().numpy()[written], exps[written])
        if n == 0:
            continue
        bare = e.scorer(n)
        bare.run()
        torch.cuda.synchronize()
        for r in range(n):                                       # one product instruction a pair, in either kernel
            m = int(bare.row_len[r])
            assert m == (pos[r] + 1) // c == int(e.path.row_len[r])
            assert torch.equal(bare.scores[r, :m], e.path.scores[r, :m])
        assert torch.equal(bare.slots.sort(1).values, e.path.slots[:n].sort(1).values)
        K, V = ref.values()
        some = sorted({0, n // 2, n - 1})
        lists = [x[x >= 0] for x in e.path.slots[some].cpu().numpy()]
        res = [attend_row(_f64(e.q[r]), K[s], V[s], d ** -0.5) for r, s in zip(some, lists)]
        check_rows(_f64(e.out[some]), _f64(e.lse[some]), res, "bf16", [len(s) for s in lists], np.abs(V).max())
        if i in keep:
            for s in (a, e):
                s.batch.release(_i32(keep[i]))


def test_two_batches_at_once_on_two_streams():
    """The calls of two batches, each on a stream of its own, overlap without a word to each other."""
    say("two streams")
    B, rows, cap, pages = 300, 4000, 4096, 3000
    steps = [Step(1, B, rows, cap, pages, 64) for _ in range(2)]
    alone = [Step(1, B, rows, cap, pages, 64) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(3):
        for j, (s, t) in enumerate(zip(steps, alone)):
            new = np.random.default_rng(10 * i + j).integers(0, 14, B)
            for x in (s, t):
                x.new.copy_(_i32(new))
                x.fill(100 * i + j)
        torch.cuda.synchronize()
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.run()
        torch.cuda.synchronize()
        for s, t in zip(steps, alone):
            t.run()
            torch.cuda.synchronize()
            want = t.results()
            for n, x in s.results().items():
                assert torch.equal(x, want[n]), (i, n)


def test_a_slot_named_twice_harms_no_other():
    """Outside the calls' preconditions: what the slot (8 bits: its page) holds is open, everything else is right."""
    say("slots twice")
    rng = np.random.default_rng(3)
    slots = np.arange(64, 64 + 150)
    slots[40] = slots[41] = slots[10]                            # page 1, three times; pages 2 and 3 are clean
    for n in (150, 2300):                                        # and among many rows: the other store kernel
        at = np.concatenate([slots, 64 * 5 + np.arange(n - 150)])
        k, v = (torch.tensor(rng.standard_normal((n, 2, 64))).bfloat16().cuda() for _ in range(2))
        cache, ref = bst.KV8Cache.empty(60, 2, 64, "cuda"), Kv8(60, 2, 64)
        bst.kv8_store(k, v, _i32(at), cache)
        ref.store(_f64(k), _f64(v), at)
        got = cache.codes.cpu().numpy()
        clean = np.setdiff1d(np.arange(60 * 64), np.arange(64, 128))
        np.testing.assert_array_equal(got[clean], ref.codes[clean])
        x = torch.tensor(rng.standard_normal((n, 128))).bfloat16().cuda()
        keys = bst.Idx4Cache.empty(60, 1, "cuda")
        bst.idx4_store(x, _i32(at), keys)
        codes, exps = quantise(_f64(x))
        once = np.isin(np.arange(n), [10, 40, 41], invert=True)
        np.testing.assert_array_equal(keys.codes.cpu().numpy()[at[once]], codes[once])
        np.testing.assert_array_equal(keys.scales.cpu().numpy()[at[once]], exps[once])
