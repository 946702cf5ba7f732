"""The whole hot path on one GPU: score -> top-k -> expand/translate, and the
attention that reads the chosen slots; and the state of a batch that they work
on, its page tables among it.

Allocates the output and workspace tensors once (torch, device memory) and
then enqueues the three C-ABI calls on the current stream.  No host
synchronisation happens inside :meth:`IndexerPath.run`.
"""
from __future__ import annotations

import torch

from . import (ATTN_WORKSPACE_BYTES, attn_slots, attn_workspace, idx_expand_translate, idx_score_decode,
               idx4_score, idx_score_prefill, idx_select_translate, idx_select_translate_planned, PagePool, pages_extend,
               pages_release, prepare_idx4_score, prepare_score, prepare_select_translate, topk_plan, topk_plan_rows,
               topk_planned_workspace, topk_select_rows, topk_workspace)


class PagedBatch:
    """Requests whose tokens live in the pages of one pool: the tables and
    lengths, kept on the GPU, and the rows of the step in hand.

    Row b of ``page_table`` (and ``kv_len``, ``held``) is request b.  After
    ``extend``, ``req_row_ptr`` and ``row_pos`` are what the scorers, the
    selection and ``attn_window`` take, and ``slots`` what ``kv4_store``,
    ``kv8_store`` and ``idx4_store`` (c = 1) take; ``tok_start`` and
    ``req_row_ptr`` are what the key compression takes, with a ring of
    ``key_ring``.  Nothing here waits for the GPU; calls on one batch belong on one
    stream."""

    def __init__(self, num_req: int, max_tokens: int, num_pages: int, num_rows: int, device):
        n = dict(dtype=torch.int32, device=device)
        self.pool = PagePool.full(num_pages, device)
        self.page_table = torch.full((num_req, max(1, -(-max_tokens // 64))), -1, **n)
        self.kv_len = torch.zeros(num_req, **n)
        self.held = torch.zeros(num_req, **n)
        self.tok_start = torch.zeros(num_req, **n)
        self.req_row_ptr = torch.zeros(num_req + 1, **n)
        self.row_pos = torch.full((num_rows,), -1, **n)
        self.slots = torch.full((num_rows,), -1, **n)

    def extend(self, new_len, stream=None):
        """Appends ``new_len`` [num_req] tokens: rows, positions, slots, pages."""
        pages_extend(self.pool, self.kv_len, self.held, new_len, self.page_table, self.req_row_ptr, self.row_pos,
                     self.slots, tok_start=self.tok_start, stream=stream)

    def key_ring(self, most_cut: int, mrope: bool = False):
        """``ring`` and ``ring_pos`` (None unless the keys have MRoPE positions) for
        the key compression of this batch, deep enough for requests that
        ``release`` cuts back to up to ``most_cut`` tokens below the most that they
        have had: the draft tokens of a step, say."""
        slots = 4
        while slots < int(most_cut) + 3:
            slots *= 2
        n, dev = self.kv_len.numel(), self.kv_len.device
        return (torch.zeros((n, slots, 128), dtype=torch.bfloat16, device=dev),
                torch.zeros((n, slots // 4, 3), dtype=torch.int32, device=dev) if mrope else None)

    def release(self, keep_len, stream=None):
        """Cuts requests back to ``keep_len`` [num_req] tokens (0: finished;
        below 0: left alone).  Compressed index keys (c = 4) come out right after
        it if the raw keys' ring is deep enough (``key_ring``)."""
        pages_release(self.pool, self.kv_len, self.held, keep_len, self.page_table, stream=stream)


class IndexerPath:
    """Buffers for one batch shape plus the three calls.

    ``inp`` is any object with the device-input fields (c, k, q, kcache,
    num_pages, page_table, req_row_ptr, row_pos, max_vis), e.g.
    ``synth.device.DeviceInputs``.  ``scorer`` is "decode" or "prefill", or
    "idx4" for 4-bit keys: ``kcache`` is then an ``Idx4Cache``.
    """

    def __init__(self, inp, scorer: str = "decode"):
        if scorer not in ("decode", "prefill", "idx4"):
            raise ValueError("scorer must be 'decode', 'prefill' or 'idx4'")
        if scorer == "idx4" and inp.kcache.c != inp.c:
            raise ValueError("the 4-bit keys are of another c")
        self.inp = inp
        self.scorer = scorer
        dev = inp.q.device
        R = int(inp.row_pos.shape[0])
        ld = max(int(inp.max_vis), 1)
        ld = (ld + 3) // 4 * 4  # 16-byte aligned rows
        self.scores = torch.empty((R, ld), dtype=torch.float32, device=dev)
        self.row_len = torch.empty(R, dtype=torch.int32, device=dev)
        self.sel = torch.empty((R, inp.k), dtype=torch.int32, device=dev)
        self.sel_count = torch.empty(R, dtype=torch.int32, device=dev)
        ld_out = inp.k * inp.c + inp.c - 1
        self.slots = torch.empty((R, ld_out), dtype=torch.int32, device=dev)
        self.pos = torch.empty((R, ld_out), dtype=torch.int32, device=dev)
        self.out_count = torch.empty(R, dtype=torch.int32, device=dev)
        self.workspace = topk_workspace(R, int(inp.max_vis), inp.k, dev)
        self.plan_buf = None          # planned selection: allocated on first use
        self.planned_workspace = None
        self.attn_ws = None           # attention over the chosen slots: {stream: workspace}, allocated on first use
        self._prepared = None

    def _prepare(self):
        """The two calls of the fused path with their arguments checked and
        marshalled once (``run`` then costs two plain C calls on the host)."""
        i = self.inp
        fn = "idx_score_decode" if self.scorer == "decode" else "idx_score_prefill"
        self._prepared = (
            prepare_idx4_score(i.q, i.kcache, i.page_table, i.req_row_ptr, i.row_pos, i.max_vis, self.scores,
                               self.row_len) if self.scorer == "idx4" else
            prepare_score(fn, i.q, i.kcache, i.num_pages, i.page_table, i.req_row_ptr, i.row_pos, i.c, i.max_vis,
                          self.scores, self.row_len),
            prepare_select_translate(self.scores, self.row_len, int(i.max_vis), i.k, i.req_row_ptr, i.row_pos,
                                     i.c, i.page_table, self.sel, self.sel_count, self.slots, self.out_count,
                                     out_pos=self.pos, workspace=self.workspace))

    def score(self, stream=None):
        i = self.inp
        if self.scorer == "idx4":
            idx4_score(i.q, i.kcache, i.page_table, i.req_row_ptr, i.row_pos, i.max_vis, self.scores, self.row_len,
                       stream=stream)
            return
        fn = idx_score_decode if self.scorer == "decode" else idx_score_prefill
        fn(i.q, i.kcache, i.num_pages, i.page_table, i.req_row_ptr, i.row_pos, i.c, i.max_vis,
           self.scores, self.row_len, stream=stream)

    def select(self, stream=None):
        topk_select_rows(self.scores, self.row_len, int(self.inp.max_vis), self.inp.k, self.sel,
                         self.sel_count, self.workspace, stream=stream)

    def expand(self, stream=None):
        i = self.inp
        idx_expand_translate(self.sel, self.sel_count, i.k, i.req_row_ptr, i.row_pos, i.c, i.page_table,
                             self.slots, self.out_count, out_pos=self.pos, stream=stream)

    def select_translate(self, stream=None):
        """Top-k and expand/translate fused in one kernel."""
        i = self.inp
        idx_select_translate(self.scores, self.row_len, int(i.max_vis), i.k, i.req_row_ptr, i.row_pos, i.c,
                             i.page_table, self.sel, self.sel_count, self.slots, self.out_count, out_pos=self.pos,
                             workspace=self.workspace, stream=stream)

    def plan(self, stream=None):
        """Builds the selection's work list from ``row_len`` (as the scorer
        wrote it); every later ``select_translate_planned`` uses it, until the
        next call here (the lengths change only with the row positions)."""
        i = self.inp
        if self.plan_buf is None:
            R, dev = int(i.row_pos.shape[0]), i.q.device
            self.plan_buf = topk_plan(R, int(i.max_vis), dev)
            self.planned_workspace = topk_planned_workspace(R, int(i.max_vis), i.k, dev)
        topk_plan_rows(self.row_len, int(i.max_vis), self.plan_buf, stream=stream)

    def select_translate_planned(self, stream=None):
        """``select_translate`` over the work list of the last ``plan``."""
        if self.plan_buf is None:
            raise RuntimeError("plan() must be called first")
        i = self.inp
        idx_select_translate_planned(self.scores, int(i.max_vis), i.k, i.req_row_ptr, i.row_pos, i.c, i.page_table,
                                     self.sel, self.sel_count, self.slots, self.out_count, self.plan_buf,
                                     out_pos=self.pos, workspace=self.planned_workspace, stream=stream)

    def bound(self, stream=None):
        """(score, select_translate) with arguments and stream fixed: each is
        one C call taking no arguments (for loops that run the step many
        times on one stream)."""
        return tuple(c.bind(stream) for c in self.prepared())

    def prepared(self):
        """(score, select_translate) as prepared calls: each takes an optional
        stream and launches with no per-call argument checking."""
        if self._prepared is None:
            self._prepare()
        return self._prepared

    def run(self, stream=None, fused: bool = True, planned: bool = False):
        """One pass of the path: score, then select + translate (fused into one
        kernel, the default) or the separate select and expand calls.
        planned: score, plan, then the planned select + translate."""
        if planned:
            self.score(stream)
            self.plan(stream)
            self.select_translate_planned(stream)
        elif fused:
            score, select_translate = self.prepared()
            score(stream)
            select_translate(stream)
        else:
            self.score(stream)
            self.select(stream)
            self.expand(stream)

    def attend(self, q, cache, out, scale=None, lse=None, stream=None):
        """Attention of the main query heads ``q`` [num_rows, q_heads,
        head_dim] over the slots of the last ``run``, read from ``cache``
        (``KV4Cache``, ``KV8Cache`` or ``KV16Cache``) into ``out``.

        Calls on different streams may overlap: each stream has a workspace of
        its own (32 MiB, kept with the path), and so has each captured call.
        ``run`` and the calls that read its slots are the caller's to order."""
        if stream is None:
            ws = self._attn_workspace(q.device)
        else:
            with torch.cuda.stream(stream):
                ws = self._attn_workspace(q.device)
        attn_slots(q, cache, self.slots, out, count=self.out_count, scale=scale, lse=lse, workspace=ws, stream=stream)

    def _attn_workspace(self, device):
        """The workspace of an attention call on the current stream."""
        if torch.cuda.is_current_stream_capturing():
            if self.attn_ws is None:
                raise RuntimeError("attend() must have run once before it is captured")
            # The graph's own memory, its counters cleared at each replay:
            # replays may overlap with other graphs and with eager calls.
            ws = torch.empty(ATTN_WORKSPACE_BYTES, dtype=torch.uint8, device=device)
            ws[:64 << 10].zero_()
            return ws
        if self.attn_ws is None:
            self.attn_ws = {}
        stream = torch._C._cuda_getCurrentRawStream(device.index)
        ws = self.attn_ws.get(stream)
        if ws is None:
            ws = self.attn_ws[stream] = attn_workspace(device)
        return ws
