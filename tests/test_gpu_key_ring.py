"""Key compression (c = 4) of requests that are cut back: the keys are those of the
tokens that were kept, for every remainder of the cut; the ring of raw keys, of
any depth, holds the newest tokens, each at its position's slot."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scoring_top_amd as bst
from attn_ref import quantise
from block_scoring_top_amd.pipeline import PagedBatch
from gpu_util import say
from more_ref import compressed_keys

pytestmark = pytest.mark.gpu

ROT, SECTIONS, THETA = 64, (16, 8, 8), 10000.0


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


class Loop:
    """Requests whose tokens are appended, compressed and cut back; ``four``: into 4-bit keys."""

    def __init__(self, B, cap, rows, most_cut, four, mrope):
        self.four, self.rows, self.pages = four, rows, B * (cap // 64 + 2)
        self.batch = PagedBatch(B, cap, self.pages, rows, "cuda")
        self.ring, self.ring_pos = self.batch.key_ring(most_cut, mrope)
        self.raw = torch.zeros((rows, 128), dtype=torch.bfloat16, device="cuda")
        self.at = torch.zeros((rows, 3), dtype=torch.int32, device="cuda") if mrope else None
        self.new, self.keep = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
        self.cache = bst.Idx4Cache.empty(self.pages, 4, "cuda")
        self.kcache = torch.zeros((self.pages * 16, 128), dtype=torch.bfloat16, device="cuda")

    def fill(self, new, keep, raw, at):
        self.new.copy_(_i32(new)), self.keep.copy_(_i32(keep))
        self.raw[:len(raw)] = torch.tensor(raw).bfloat16().cuda()
        if self.at is not None:
            self.at[:len(at)] = _i32(at)

    def step(self):
        b = self.batch
        b.extend(self.new)
        head = (self.raw, b.req_row_ptr, b.tok_start, self.at, self.rows, ROT, SECTIONS, THETA, self.ring, self.ring_pos,
                b.page_table)
        if self.four:
            bst.idx4_compress_store(*head, self.cache)
        else:
            bst.idx_compress_store(*head, self.kcache, self.pages)
        b.release(self.keep)

    def results(self):
        return [self.batch.kv_len, self.batch.page_table, self.ring, self.cache.codes, self.cache.scales, self.kcache] + (
            [] if self.ring_pos is None else [self.ring_pos])


def _steps(rng, B, draft, most_cut, n):
    """Per step: new tokens of each request, what is kept after it (-1: all), raw keys and positions; the tokens that each
    request has at the end, as indexes into them.  A cut goes back up to ``most_cut`` tokens from the longest that the
    request has been, into the tokens of earlier steps too; some requests finish, and others begin in their place."""
    tokens, high, out, total, cuts = [[] for _ in range(B)], np.zeros(B, int), [], 0, set()
    for i in range(n):
        new = rng.integers(1, draft + 1, B) if i else rng.integers(1, 90, B)
        new[rng.random(B) < 0.1] = 0
        keep = np.full(B, -1)
        for b in range(B):
            tokens[b] += range(total, total + new[b])
            total += new[b]
            high[b] = max(high[b], len(tokens[b]))
            low = max(0, high[b] - most_cut)
            if i and rng.random() < 0.04:
                keep[b], tokens[b], high[b] = 0, [], 0
            elif i and rng.random() < 0.7 and len(tokens[b]) > low:
                keep[b] = rng.integers(low, len(tokens[b]))
                cuts.add((len(tokens[b]) % 4, keep[b] % 4))
                tokens[b] = tokens[b][:keep[b]]
        out.append((new, keep, rng.standard_normal((new.sum(), 128)), rng.integers(0, 3000, (new.sum(), 3))))
    assert len(cuts) == 16                                       # every remainder, from every remainder
    return out, tokens


@pytest.mark.parametrize("mrope", [False, True])
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("draft,most_cut", [(6, 6), (2, 5), (13, 13), (7, 29)])
def test_keys_after_cuts_are_of_the_kept_tokens(draft, most_cut, four, mrope):
    """4-bit keys against 64 bits, codes and scales exact (no element of these fixed inputs is near a tie); bf16 keys
    against one call that is given the kept tokens alone, exact: the same operations on the same keys."""
    say(f"key ring draft={draft} most_cut={most_cut} four={four} mrope={mrope}")
    rng = np.random.default_rng(100 * draft + most_cut)
    B, cap = 16, 1000
    steps, tokens = _steps(rng, B, draft, most_cut, 26)
    s = Loop(B, cap, B * 100, most_cut, four, mrope)
    for x in steps:
        s.fill(*x)
        s.step()
    torch.cuda.synchronize()
    n = np.array([len(t) for t in tokens])
    assert s.batch.kv_len.tolist() == n.tolist() and (n > 20).any()
    raw = torch.tensor(np.concatenate([x[2] for x in steps])).bfloat16()
    where = np.concatenate([x[3] for x in steps])
    table = s.batch.page_table.cpu().numpy()
    at = np.concatenate([table[b, np.arange(n[b] // 4) // 16] * 16 + np.arange(n[b] // 4) % 16 for b in range(B)])
    if four:
        keys = []
        for b in range(B):
            ids = np.array(tokens[b], int)[:n[b] // 4 * 4].reshape(-1, 4)
            first = where[ids[:, 0]] if mrope else 4 * np.arange(len(ids))[:, None].repeat(3, 1)
            if len(ids):
                keys.append(compressed_keys(raw.double().numpy()[ids], first, ROT, SECTIONS, THETA))
        codes, scales = quantise(np.concatenate(keys))
        np.testing.assert_array_equal(s.cache.codes.cpu().numpy()[at], codes)
        np.testing.assert_array_equal(s.cache.scales.cpu().numpy()[at], scales)
        return
    ids = np.concatenate(tokens).astype(int)
    want = torch.zeros_like(s.kcache)
    bst.idx_compress_store(raw[ids].cuda(), _i32(np.concatenate([[0], n.cumsum()])), _i32(np.zeros(B)),
                           _i32(where[ids]) if mrope else None, int(n.max()), ROT, SECTIONS, THETA,
                           torch.zeros((B, 4, 128), dtype=torch.bfloat16, device="cuda"),
                           torch.zeros((B, 3), dtype=torch.int32, device="cuda"), s.batch.page_table, want, s.pages)
    at = torch.from_numpy(at).long().cuda()
    assert torch.equal(s.kcache[at], want[at]) and want[at].any(1).all()


@pytest.mark.parametrize("four", [False, True])
def test_cuts_in_a_captured_step(four):
    """A step with its compression and its cut, captured once and replayed with other tokens, like an eager one."""
    say(f"key ring captured four={four}")
    steps, _ = _steps(np.random.default_rng(5), 16, 6, 9, 20)
    a, e = (Loop(16, 600, 16 * 90, 9, four, True) for _ in range(2))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a.step()                                                 # no tokens
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step()
    torch.cuda.synchronize()
    for x in steps:
        a.fill(*x), e.fill(*x)
        e.step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip(a.results(), e.results()):
            assert torch.equal(got, want)


@pytest.mark.parametrize("slots", [4, 8, 64, 1024])
@pytest.mark.parametrize("mrope", [False, True])
def test_the_ring_holds_the_newest_tokens(slots, mrope):
    """As if every new token were written in the order of positions, and nothing else."""
    say(f"key ring slots={slots} mrope={mrope}")
    rng = np.random.default_rng(slots)
    start, new = np.array([0, 3, 61, 7, 1 << 20, 2**31 - 700, 5]), np.array([1, 6, 1500, 0, 130, 600, 9])
    B, T, most = len(start), new.sum(), 1400
    ptr = np.concatenate([[0], new.cumsum()])
    raw = torch.tensor(rng.standard_normal((T, 128))).bfloat16()
    at = rng.integers(0, 3000, (T, 3))
    ring = torch.tensor(rng.standard_normal((B, slots, 128))).bfloat16()
    pos = rng.integers(0, 99, (B, slots // 4, 3))
    r, p = ring.cuda(), _i32(pos)
    kc = torch.zeros((16, 128), dtype=torch.bfloat16, device="cuda")
    for cache in ("16", "4"):
        r.copy_(ring), p.copy_(_i32(pos))
        head = (raw.cuda(), _i32(ptr), _i32(start), _i32(at) if mrope else None, most, ROT, SECTIONS, THETA, r, p,
                _i32([[-1]] * B))
        if cache == "4":
            bst.idx4_compress_store(*head, bst.Idx4Cache.empty(1, 4, "cuda"))
        else:
            bst.idx_compress_store(*head, kc, 1)
        want, want_pos = ring.clone(), pos.copy()
        for b in range(B):
            for j in range(min(new[b], most)):
                q = int(start[b]) + j
                want[b, q % slots] = raw[ptr[b] + j]
                if q % 4 == 0:
                    want_pos[b, q // 4 % (slots // 4)] = at[ptr[b] + j] if mrope else q
        assert torch.equal(r.cpu(), want)
        np.testing.assert_array_equal(p.cpu().numpy(), want_pos)
    assert not kc.any()
