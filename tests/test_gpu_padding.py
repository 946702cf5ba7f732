"""Rows behind the last request's, after steps that had more: no length, nothing
selected, no slots, whichever scorer and selection, eager and captured."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scoring_top_amd as bst
from block_scoring_top_amd.pipeline import IndexerPath, PagedBatch
from gpu_util import say

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def _path(scorer, c, batch, rows, cap, pages, k, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kc = torch.randn((pages * 64 // c, 128), generator=g, device="cuda").bfloat16()
    if scorer == "idx4":
        keys = bst.Idx4Cache.empty(pages, c, "cuda")
        bst.idx4_store(kc, torch.arange(len(kc), dtype=torch.int32, device="cuda"), keys)
        kc = keys
    q = torch.randn((rows, 4, 128), generator=g, device="cuda").bfloat16()
    return IndexerPath(type("Inputs", (), dict(c=c, k=k, q=q, kcache=kc, num_pages=pages, page_table=batch.page_table,
                                               req_row_ptr=batch.req_row_ptr, row_pos=batch.row_pos, max_vis=cap // c))(), scorer)


def _outputs(p):
    return dict(row_len=p.row_len, sel=p.sel, sel_count=p.sel_count, slots=p.slots, pos=p.pos, out_count=p.out_count)


# rows on average, with the padding: those of each kernel of each scorer
@pytest.mark.parametrize("B,rows", [(700, 700), (300, 600), (64, 400), (9, 500), (1, 3000), (3, 20000)])
@pytest.mark.parametrize("scorer,c", [("decode", 4), ("decode", 1), ("prefill", 4), ("idx4", 4), ("idx4", 1)])
@pytest.mark.parametrize("how", ["fused", "apart", "planned"])
def test_nothing_is_left_of_a_fuller_step(scorer, c, B, rows, how):
    say(f"padding {scorer} c={c} B={B} rows={rows} {how}")
    cap, k = 1024, 32
    pages = B * 17
    batch = PagedBatch(B, cap, pages, rows, "cuda")
    p = _path(scorer, c, batch, rows, cap, pages, k, B)
    n = min(rows // B, 500)
    steps = [[n] * B, [max(1, n // 3)] * (B - 1) + [1], [0] * B, [1] + [0] * (B - 1)]
    kw = dict(fused=how == "fused", planned=how == "planned")
    done = np.zeros(B, int)
    for new in steps:
        for x in (p.row_len, p.sel_count, p.out_count):          # what memory may hold
            x.fill_(cap // c if new is steps[0] else 7)
        batch.extend(_i32(new))
        p.run(**kw)
        torch.cuda.synchronize()
        t = sum(new)
        out = _outputs(p)
        assert int(batch.req_row_ptr[-1]) == t
        for name in ("row_len", "sel_count", "out_count"):
            assert not out[name][t:].any(), name
        for name in ("sel", "slots", "pos"):
            assert (out[name][t:] == -1).all(), name
        pos = np.concatenate([np.arange(a, a + m) for a, m in zip(done, new)])
        done += new
        np.testing.assert_array_equal(out["row_len"][:t].cpu().numpy(), (pos + 1) // c)
        np.testing.assert_array_equal(out["sel_count"][:t].cpu().numpy(), np.minimum((pos + 1) // c, k))


@pytest.mark.parametrize("scorer", ["decode", "prefill", "idx4"])
def test_replayed_steps(scorer):
    """One captured step, replayed with fewer rows than before and with more; long rows, whose selection is split."""
    say(f"padding captured {scorer}")
    B, rows, cap, c, k = 3, 40, 40000, 1, 64
    pages = B * 626
    batch = PagedBatch(B, cap, pages, rows, "cuda")
    p = _path(scorer, c, batch, rows, cap, pages, k, 1)
    fill = PagedBatch(B, cap, pages, 3 * 39000, "cuda")          # the same batch with room for the prompts
    for name in ("pool", "page_table", "kv_len", "held"):
        setattr(fill, name, getattr(batch, name))
    fill.extend(_i32([39000, 35000, 500]))
    new = torch.zeros(B, dtype=torch.int32, device="cuda")

    def step():
        batch.extend(new)
        p.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    torch.cuda.synchronize()
    for n in ([30, 5, 5], [1, 1, 1], [0, 0, 0], [10, 0, 20], [0, 1, 0]):
        new.copy_(_i32(n))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        out, t = _outputs(p), sum(n)
        for name in ("row_len", "sel_count", "out_count"):
            assert not out[name][t:].any() and (out[name][:t] > 0).all(), (n, name)
        for name in ("sel", "slots", "pos"):
            assert (out[name][t:] == -1).all(), (n, name)
