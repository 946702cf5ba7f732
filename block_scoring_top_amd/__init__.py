"""MI355X-native sparse-attention indexer hot path.

Thin Python binding over ``libblockscore.so`` (C ABI in ``include/blockscore.h``).
Every function here only marshals torch tensors into the C call: it checks
dtypes, devices and contiguity, takes raw device pointers and the current HIP
stream, and raises if the library returns an error.  All computation runs in
the HIP kernels; there is no CPU fallback.  If the library is not built this
module raises on first use.

Steps (same names as the C ABI):
  idx_score_decode / idx_score_prefill  ->  topk_select_rows  ->  idx_expand_translate
  (idx_select_translate: the last two in one kernel; topk_plan_rows +
  idx_select_translate_planned: the same over a work list built once per step
  from the row lengths; idx_expand_translate_shared: the expansion of a
  selection reused across speculative draft steps)
What consumes the chosen slots:
  kv4_store / kv4_load (a 4-bit KV cache, written and read back) and
  attn_slots / attn_window (attention over a selection's slots, and over a
  sliding window plus the first tokens; 16-bit pools, the 4-bit cache or the
  8-bit one that kv8_store / kv8_load write and read)
The index keys in 4 bits: idx4_store / idx4_compress_store / idx4_load, scored
  by idx4_score in place of the first step.
The tables, positions and slots that these calls take, kept on the GPU:
  pages_extend / pages_release.
"""
from __future__ import annotations

import ctypes as C
import math
import os
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libblockscore.so")

HEADS = 4
DIM = 128
PAGE_TOKENS = 64
KMAX = 2048
NOALLOC_SCRATCH_BYTES = 8 << 20  # BS_NOALLOC_SCRATCH_BYTES
ATTN_WORKSPACE_BYTES = (32 << 20) + (64 << 10)  # BS_ATTN_WORKSPACE_BYTES

_lib = None


class BlockScoreError(RuntimeError):
    pass


def lib():
    """Loads the HIP library (built by ``block_scoring_top_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise BlockScoreError(
                f"{LIB_PATH} is missing: build it with `python -m block_scoring_top_amd.build` "
                "(or __graft_entry__.build()); there is no CPU fallback")
        L = C.CDLL(LIB_PATH)
        P, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
        score_args = [P, P, i64, P, i32, P, i32, P, i32, i32, i32, P, i64, P, P]
        for name in ("idx_score_decode", "idx_score_prefill"):
            f = getattr(L, name)
            f.argtypes = score_args
            f.restype = C.c_int
        L.topk_workspace_bytes.argtypes = [i32, i32, i32]
        L.topk_workspace_bytes.restype = C.c_size_t
        L.topk_select_rows.argtypes = [P, i64, P, i32, i32, i32, P, P, P, C.c_size_t, P]
        L.topk_select_rows.restype = C.c_int
        L.idx_expand_translate.argtypes = [P, P, i32, P, i32, P, i32, i32, P, i32, P, P, P, i32, P]
        L.idx_expand_translate.restype = C.c_int
        L.idx_expand_translate_shared.argtypes = [P, P, i32, P, i32, P, P, i32, i32, i32, P, i32, P, P, P, i32, P]
        L.idx_expand_translate_shared.restype = C.c_int
        L.idx_select_translate.argtypes = [P, i64, P, i32, i32, i32, P, i32, P, i32, P, i32, P, P, P, P, P, i32,
                                           P, C.c_size_t, P]
        L.idx_select_translate.restype = C.c_int
        L.idx_select_translate_noalloc.argtypes = [P, i64, P, i32, i32, i32, P, i32, P, i32, P, i32, P, P, P, P, P,
                                                   i32, P]
        L.idx_select_translate_noalloc.restype = C.c_int
        L.topk_plan_bytes.argtypes = [i32, i32]
        L.topk_plan_bytes.restype = C.c_size_t
        L.topk_planned_workspace_bytes.argtypes = [i32, i32, i32]
        L.topk_planned_workspace_bytes.restype = C.c_size_t
        L.topk_plan_rows.argtypes = [P, i32, i32, P, C.c_size_t, P]
        L.topk_plan_rows.restype = C.c_int
        L.idx_select_translate_planned.argtypes = [P, i64, i32, i32, i32, P, i32, P, i32, P, i32, P, P, P, P, P,
                                                   i32, P, C.c_size_t, P, C.c_size_t, P]
        L.idx_select_translate_planned.restype = C.c_int
        L.idx_compress_store.argtypes = [P, i32, P, P, P, i32, i32, i32, i32, i32, i32, C.c_double, P, P, P, i32,
                                         P, i64, P]
        L.idx_compress_store.restype = C.c_int
        L.idx_compress_store_ring.argtypes = [P, i32, P, P, P, i32, i32, i32, i32, i32, i32, C.c_double, P, P, i32, P,
                                              i32, P, i64, P]
        L.idx_compress_store_ring.restype = C.c_int
        L.kv4_store.argtypes = [P, P, i32, i64, i64, P, i32, i32, i32, P, P, i64, P]
        L.kv4_store.restype = C.c_int
        L.kv4_load.argtypes = [P, P, i64, P, i32, i32, i32, P, P, i32, i64, i64, P]
        L.kv4_load.restype = C.c_int
        L.kv8_store.argtypes = L.kv4_store.argtypes
        L.kv8_store.restype = C.c_int
        L.kv8_load.argtypes = L.kv4_load.argtypes
        L.kv8_load.restype = C.c_int
        L.idx4_store.argtypes = [P, i32, i64, P, i32, P, P, i64, P]
        L.idx4_store.restype = C.c_int
        L.idx4_load.argtypes = [P, P, i64, P, i32, P, i32, i64, P]
        L.idx4_load.restype = C.c_int
        L.idx4_compress_store.argtypes = [P, i32, P, P, P, i32, i32, i32, i32, i32, i32, C.c_double, P, P, P, i32,
                                          P, P, i64, P]
        L.idx4_compress_store.restype = C.c_int
        L.idx4_compress_store_ring.argtypes = [P, i32, P, P, P, i32, i32, i32, i32, i32, i32, C.c_double, P, P, i32, P,
                                               i32, P, P, i64, P]
        L.idx4_compress_store_ring.restype = C.c_int
        L.idx4_score.argtypes = [P, P, P, i64, P, i32, P, i32, P, i32, i32, i32, P, i64, P, P]
        L.idx4_score.restype = C.c_int
        pages_args = [P, P, P, i32, P, i32, P, i32, P, P, P, P]
        L.pages_extend.argtypes = [*pages_args, P, P, P, P, i32, P]
        L.pages_extend.restype = C.c_int
        L.pages_release.argtypes = [*pages_args, P]
        L.pages_release.restype = C.c_int
        attn_args = [P, i32, i64, i32, i32, i32, i32, P, P, i32, i64, i64]
        L.attn_slots.argtypes = [*attn_args, P, i32, P, C.c_float, P, i64, P, P, C.c_size_t, P]
        L.attn_slots.restype = C.c_int
        L.attn_window.argtypes = [*attn_args, P, i32, P, i32, P, i32, i32, i32, C.c_float, P, i64, P, P, C.c_size_t, P]
        L.attn_window.restype = C.c_int
        L.bs_status_string.argtypes = [C.c_int]
        L.bs_status_string.restype = C.c_char_p
        L.bs_abi_version.argtypes = []
        L.bs_abi_version.restype = C.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().bs_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != 0:
        raise BlockScoreError(f"{what}: {status_string(status)} ({status})")


def _ptr(t: Optional[torch.Tensor], dtypes, name: str, device: Optional[torch.device] = None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return C.c_void_p(t.data_ptr())


def _stream(stream, device) -> C.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return C.c_void_p(s.cuda_stream)


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_I32 = (torch.int32,)
_F32 = (torch.float32,)


def _score_args(q, kcache, num_pages, page_table, req_row_ptr, row_pos, c, max_vis, scores, row_len=None):
    """Checked argument tuple of a scorer call (all but the stream)."""
    dev = q.device
    num_rows = int(row_pos.shape[0])
    num_req = int(req_row_ptr.shape[0]) - 1
    if q.numel() != num_rows * HEADS * DIM:
        raise ValueError("q must hold num_rows x 4 x 128 values")
    if scores.dim() != 2 or scores.shape[0] != num_rows:
        raise ValueError("scores must be [num_rows, ld]")
    if row_len is not None and row_len.numel() != num_rows:
        raise ValueError("row_len must hold num_rows entries")
    per_page = PAGE_TOKENS // int(c) if int(c) in (1, 4) else 1
    if kcache is not None and kcache.numel() < int(num_pages) * per_page * DIM:
        raise ValueError("kcache holds fewer than num_pages pages")
    return (_ptr(q, _BF16, "q", dev), _ptr(kcache, _BF16, "kcache", dev), int(num_pages),
            _ptr(page_table, _I32, "page_table", dev), int(page_table.shape[1]),
            _ptr(req_row_ptr, _I32, "req_row_ptr", dev), num_req,
            _ptr(row_pos, _I32, "row_pos", dev), num_rows, int(c), int(max_vis),
            _ptr(scores, _F32, "scores", dev), int(scores.stride(0)),
            _ptr(row_len, _I32, "row_len", dev))


def _score(fn: str, q, kcache, num_pages, page_table, req_row_ptr, row_pos, c, max_vis, scores,
           row_len=None, stream=None):
    args = _score_args(q, kcache, num_pages, page_table, req_row_ptr, row_pos, c, max_vis, scores, row_len)
    _check(getattr(lib(), fn)(*args, _stream(stream, q.device)), fn)


def idx_score_decode(q, kcache, num_pages, page_table, req_row_ptr, row_pos, c, max_vis, scores,
                     row_len=None, stream=None):
    """Paged decode/verify scorer.  See ``idx_score_decode`` in blockscore.h."""
    _score("idx_score_decode", q, kcache, num_pages, page_table, req_row_ptr, row_pos, c, max_vis,
           scores, row_len, stream)


def idx_score_prefill(q, kcache, num_pages, page_table, req_row_ptr, row_pos, c, max_vis, scores,
                      row_len=None, stream=None):
    """Prefill scorer on the matrix cores.  See ``idx_score_prefill`` in blockscore.h."""
    _score("idx_score_prefill", q, kcache, num_pages, page_table, req_row_ptr, row_pos, c, max_vis,
           scores, row_len, stream)


def topk_workspace_bytes(num_rows: int, max_len: int, k: int) -> int:
    return int(lib().topk_workspace_bytes(int(num_rows), int(max_len), int(k)))


def topk_workspace(num_rows: int, max_len: int, k: int, device) -> Optional[torch.Tensor]:
    """A zero-filled workspace of the size the call needs (None if none)."""
    n = topk_workspace_bytes(num_rows, max_len, k)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def _topk_args(scores, row_len, max_len, k, sel, sel_count, workspace=None):
    """Checked argument tuple of a ``topk_select_rows`` call (all but the stream)."""
    dev = scores.device
    R = int(scores.shape[0])
    if sel.dim() != 2 or sel.shape[0] != R or sel.shape[1] != k:
        raise ValueError("sel must be [num_rows, k]")
    if sel_count.numel() != R or row_len.numel() != R:
        raise ValueError("row_len and sel_count must hold num_rows entries")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return (_ptr(scores, _F32, "scores", dev), int(scores.stride(0)), _ptr(row_len, _I32, "row_len", dev), R,
            int(max_len), int(k), _ptr(sel, _I32, "sel", dev), _ptr(sel_count, _I32, "sel_count", dev),
            _ptr(workspace, (torch.uint8,), "workspace", dev), ws_bytes)


def topk_select_rows(scores, row_len, max_len, k, sel, sel_count, workspace=None, stream=None):
    """Exact top-k per FP32 row.  See ``topk_select_rows`` in blockscore.h."""
    args = _topk_args(scores, row_len, max_len, k, sel, sel_count, workspace)
    _check(lib().topk_select_rows(*args, _stream(stream, scores.device)), "topk_select_rows")


def idx_expand_translate(sel, sel_count, k, req_row_ptr, row_pos, c, page_table, out_slots, out_count,
                         out_pos=None, stream=None):
    """Expand, append pending, translate.  See ``idx_expand_translate`` in blockscore.h."""
    dev = sel.device
    R = int(row_pos.shape[0])
    if sel.dim() != 2 or sel.shape[0] != R or sel.shape[1] != k:
        raise ValueError("sel must be [num_rows, k]")
    if out_slots.dim() != 2 or out_slots.shape[0] != R:
        raise ValueError("out_slots must be [num_rows, ld_out]")
    if out_pos is not None and out_pos.shape != out_slots.shape:
        raise ValueError("out_pos must match out_slots")
    st = lib().idx_expand_translate(
        _ptr(sel, _I32, "sel", dev), _ptr(sel_count, _I32, "sel_count", dev), int(k),
        _ptr(req_row_ptr, _I32, "req_row_ptr", dev), int(req_row_ptr.shape[0]) - 1,
        _ptr(row_pos, _I32, "row_pos", dev), R, int(c),
        _ptr(page_table, _I32, "page_table", dev), int(page_table.shape[1]),
        _ptr(out_slots, _I32, "out_slots", dev), _ptr(out_pos, _I32, "out_pos", dev),
        _ptr(out_count, _I32, "out_count", dev), int(out_slots.stride(0)), _stream(stream, dev))
    _check(st, "idx_expand_translate")


def _expand_shared_args(sel, sel_count, k, req_row_ptr, row_pos, row_pos_now, c, max_advance, page_table,
                        out_slots, out_count, out_pos=None):
    """Checked argument tuple of an ``idx_expand_translate_shared`` call (all but the stream)."""
    dev = sel.device
    R = int(row_pos.shape[0])
    if sel.dim() != 2 or sel.shape[0] != R or sel.shape[1] != k:
        raise ValueError("sel must be [num_rows, k]")
    if row_pos_now.numel() != R or sel_count.numel() != R:
        raise ValueError("row_pos_now and sel_count must hold num_rows entries")
    if out_slots.dim() != 2 or out_slots.shape[0] != R:
        raise ValueError("out_slots must be [num_rows, ld_out]")
    if out_pos is not None and out_pos.shape != out_slots.shape:
        raise ValueError("out_pos must match out_slots")
    return (_ptr(sel, _I32, "sel", dev), _ptr(sel_count, _I32, "sel_count", dev), int(k),
            _ptr(req_row_ptr, _I32, "req_row_ptr", dev), int(req_row_ptr.shape[0]) - 1,
            _ptr(row_pos, _I32, "row_pos", dev), _ptr(row_pos_now, _I32, "row_pos_now", dev), R, int(c),
            int(max_advance), _ptr(page_table, _I32, "page_table", dev), int(page_table.shape[1]),
            _ptr(out_slots, _I32, "out_slots", dev), _ptr(out_pos, _I32, "out_pos", dev),
            _ptr(out_count, _I32, "out_count", dev), int(out_slots.stride(0)))


def idx_expand_translate_shared(sel, sel_count, k, req_row_ptr, row_pos, row_pos_now, c, max_advance, page_table,
                                out_slots, out_count, out_pos=None, stream=None):
    """Expansion of a selection reused across draft steps (IndexShare).  See
    ``idx_expand_translate_shared`` in blockscore.h."""
    args = _expand_shared_args(sel, sel_count, k, req_row_ptr, row_pos, row_pos_now, c, max_advance, page_table,
                               out_slots, out_count, out_pos)
    _check(lib().idx_expand_translate_shared(*args, _stream(stream, sel.device)), "idx_expand_translate_shared")


def _select_translate_args(scores, row_len, max_len, k, req_row_ptr, row_pos, c, page_table, sel, sel_count,
                           out_slots, out_count, out_pos=None, workspace=None):
    """Checked argument tuple of an ``idx_select_translate`` call (all but the stream)."""
    dev = scores.device
    R = int(scores.shape[0])
    if sel.dim() != 2 or sel.shape[0] != R or sel.shape[1] != k:
        raise ValueError("sel must be [num_rows, k]")
    if sel_count.numel() != R or row_pos.numel() != R or (row_len is not None and row_len.numel() != R):
        raise ValueError("row_len, row_pos and sel_count must hold num_rows entries")
    if out_slots.dim() != 2 or out_slots.shape[0] != R:
        raise ValueError("out_slots must be [num_rows, ld_out]")
    if out_pos is not None and out_pos.shape != out_slots.shape:
        raise ValueError("out_pos must match out_slots")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return (_ptr(scores, _F32, "scores", dev), int(scores.stride(0)), _ptr(row_len, _I32, "row_len", dev), R,
            int(max_len), int(k), _ptr(req_row_ptr, _I32, "req_row_ptr", dev), int(req_row_ptr.shape[0]) - 1,
            _ptr(row_pos, _I32, "row_pos", dev), int(c), _ptr(page_table, _I32, "page_table", dev),
            int(page_table.shape[1]), _ptr(sel, _I32, "sel", dev), _ptr(sel_count, _I32, "sel_count", dev),
            _ptr(out_slots, _I32, "out_slots", dev), _ptr(out_pos, _I32, "out_pos", dev),
            _ptr(out_count, _I32, "out_count", dev), int(out_slots.stride(0)),
            _ptr(workspace, (torch.uint8,), "workspace", dev), ws_bytes)


def idx_select_translate(scores, row_len, max_len, k, req_row_ptr, row_pos, c, page_table, sel, sel_count,
                         out_slots, out_count, out_pos=None, workspace=None, stream=None):
    """Top-k and expand/translate in one kernel.  See ``idx_select_translate`` in blockscore.h."""
    args = _select_translate_args(scores, row_len, max_len, k, req_row_ptr, row_pos, c, page_table, sel,
                                  sel_count, out_slots, out_count, out_pos, workspace)
    _check(lib().idx_select_translate(*args, _stream(stream, scores.device)), "idx_select_translate")


def idx_select_translate_noalloc(scores, row_len, max_len, k, req_row_ptr, row_pos, c, page_table, sel, sel_count,
                                 out_slots, out_count, out_pos=None, stream=None):
    """``idx_select_translate`` without a workspace (static device scratch of
    NOALLOC_SCRATCH_BYTES per GPU).  See ``idx_select_translate_noalloc`` in
    blockscore.h."""
    args = _select_translate_args(scores, row_len, max_len, k, req_row_ptr, row_pos, c, page_table, sel,
                                  sel_count, out_slots, out_count, out_pos, None)[:-2]
    _check(lib().idx_select_translate_noalloc(*args, _stream(stream, scores.device)), "idx_select_translate_noalloc")


def topk_plan_bytes(num_rows: int, max_len: int) -> int:
    return int(lib().topk_plan_bytes(int(num_rows), int(max_len)))


def topk_planned_workspace_bytes(num_rows: int, max_len: int, k: int) -> int:
    return int(lib().topk_planned_workspace_bytes(int(num_rows), int(max_len), int(k)))


def topk_plan(num_rows: int, max_len: int, device) -> torch.Tensor:
    """Storage for a plan (int32, uninitialised: ``topk_plan_rows`` fills it)."""
    n = topk_plan_bytes(num_rows, max_len)
    return torch.empty(max(1, (n + 3) // 4), dtype=torch.int32, device=device)


def topk_planned_workspace(num_rows: int, max_len: int, k: int, device) -> Optional[torch.Tensor]:
    """A zero-filled workspace for ``idx_select_translate_planned`` (None if none)."""
    n = topk_planned_workspace_bytes(num_rows, max_len, k)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def _plan_args(row_len, max_len, plan):
    dev = row_len.device
    return (_ptr(row_len, _I32, "row_len", dev), int(row_len.numel()), int(max_len), _ptr(plan, _I32, "plan", dev),
            plan.numel() * plan.element_size())


def topk_plan_rows(row_len, max_len, plan, stream=None):
    """Build the selection's work list from the row lengths.  See
    ``topk_plan_rows`` in blockscore.h."""
    _check(lib().topk_plan_rows(*_plan_args(row_len, max_len, plan), _stream(stream, row_len.device)),
           "topk_plan_rows")


def _select_translate_planned_args(scores, max_len, k, req_row_ptr, row_pos, c, page_table, sel, sel_count,
                                   out_slots, out_count, plan, out_pos=None, workspace=None):
    # The argument tuple of idx_select_translate with row_len taken out and the
    # plan put before the workspace.
    a = _select_translate_args(scores, None, max_len, k, req_row_ptr, row_pos, c, page_table, sel, sel_count,
                               out_slots, out_count, out_pos, workspace)
    return (*a[:2], *a[3:18], _ptr(plan, _I32, "plan", scores.device), plan.numel() * plan.element_size(), *a[18:])


def idx_select_translate_planned(scores, max_len, k, req_row_ptr, row_pos, c, page_table, sel, sel_count,
                                 out_slots, out_count, plan, out_pos=None, workspace=None, stream=None):
    """``idx_select_translate`` over the work list of a plan (the plan's row
    lengths).  See ``idx_select_translate_planned`` in blockscore.h."""
    args = _select_translate_planned_args(scores, max_len, k, req_row_ptr, row_pos, c, page_table, sel, sel_count,
                                          out_slots, out_count, plan, out_pos, workspace)
    _check(lib().idx_select_translate_planned(*args, _stream(stream, scores.device)), "idx_select_translate_planned")


def _compress_head(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok, rotary_dim, sections, theta, ring, ring_pos,
                   page_table):
    """The checked arguments that both compressing calls begin with (the C calls
    with a ring of any depth, which its shape gives)."""
    dev = k_raw.device
    T = int(k_raw.shape[0])
    B = int(req_tok_ptr.shape[0]) - 1
    if k_raw.dim() != 2 or k_raw.shape[1] != 128:
        raise ValueError("k_raw must be [num_tok, 128]")
    if tok_start.numel() != B or ring.dim() != 3 or ring.shape[0] != B or ring.shape[1] < 4 or ring.shape[2] != 128:
        raise ValueError("tok_start must hold num_req entries and ring be [num_req, ring_slots, 128]")
    slots = _size(ring.shape[1])
    if mrope_pos is not None and mrope_pos.shape != (T, 3):
        raise ValueError("mrope_pos must be [num_tok, 3]")
    if ring_pos is not None and ring_pos.shape != (B, slots // 4, 3) and (slots > 4 or ring_pos.shape != (B, 3)):
        raise ValueError("ring_pos must be [num_req, ring_slots / 4, 3]")
    sec = [int(v) for v in sections]
    if len(sec) != 3:
        raise ValueError("sections must hold 3 entries (t, h, w)")
    return (_ptr(k_raw, _BF16, "k_raw", dev), T, _ptr(req_tok_ptr, _I32, "req_tok_ptr", dev),
            _ptr(tok_start, _I32, "tok_start", dev), _ptr(mrope_pos, _I32, "mrope_pos", dev), B, int(max_tok),
            int(rotary_dim), sec[0], sec[1], sec[2], float(theta), _ptr(ring, _BF16, "ring", dev),
            _ptr(ring_pos, _I32, "ring_pos", dev), slots, _ptr(page_table, _I32, "page_table", dev),
            int(page_table.shape[1]))


def _compress_args(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok, rotary_dim, sections, theta, ring,
                   ring_pos, page_table, kcache, num_pages):
    """Checked argument tuple of an ``idx_compress_store_ring`` call (all but the stream)."""
    if kcache.dim() != 2 or kcache.shape[1] != 128 or kcache.shape[0] < 16 * int(num_pages):
        raise ValueError("kcache must be [>= num_pages * 16, 128]")
    return (*_compress_head(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok, rotary_dim, sections, theta, ring,
                            ring_pos, page_table), _ptr(kcache, _BF16, "kcache", k_raw.device), int(num_pages))


def idx_compress_store(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok, rotary_dim, sections, theta, ring,
                       ring_pos, page_table, kcache, num_pages, stream=None):
    """Compress new raw index keys into the c = 4 key cache (and update the
    rings).  ``ring`` [num_req, ring_slots, 128], ``ring_pos`` [num_req,
    ring_slots / 4, 3] or None: 4 slots for requests that only grow, more (a power
    of two, at least the tokens cut off + 3) for requests that are cut back.  See
    ``idx_compress_store`` and ``idx_compress_store_ring`` in blockscore.h."""
    args = _compress_args(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok, rotary_dim, sections, theta, ring,
                          ring_pos, page_table, kcache, num_pages)
    _check(lib().idx_compress_store_ring(*args, _stream(stream, k_raw.device)), "idx_compress_store")


_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # bs_dtype
_U8 = (torch.uint8,)
_CODES8 = (torch.uint8, torch.float8_e4m3fn)


class KV4Cache:
    """A 4-bit KV cache (layout: ``kv4_store`` in blockscore.h): ``codes``
    uint8 [slots, kv_heads, 2, head_dim / 2] and ``scales`` uint8 [slots,
    kv_heads, 2, head_dim / 32], contiguous, ``slots`` a multiple of 64."""

    form = 1  # BS_KV_4

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dim() != 4 or codes.shape[2] != 2 or codes.shape[0] % PAGE_TOKENS:
            raise ValueError("codes must be [num_pages * 64, kv_heads, 2, head_dim / 2]")
        self.codes, self.scales = codes, scales
        self.kv_heads, self.head_dim = int(codes.shape[1]), 2 * int(codes.shape[3])
        self.num_pages = int(codes.shape[0]) // PAGE_TOKENS
        if scales.shape != (codes.shape[0], self.kv_heads, 2, self.head_dim // 32):
            raise ValueError("scales must be [num_pages * 64, kv_heads, 2, head_dim / 32]")
        self.device = codes.device

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, head_dim: int, device) -> "KV4Cache":
        """Storage for ``num_pages`` pages (every slot reads back as zeros)."""
        n = int(num_pages) * PAGE_TOKENS
        return cls(torch.zeros((n, kv_heads, 2, head_dim // 2), dtype=torch.uint8, device=device),
                   torch.full((n, kv_heads, 2, head_dim // 32), 127, dtype=torch.uint8, device=device))

    def _args(self, dtype, dev):
        return _ptr(self.codes, _U8, "codes", dev), _ptr(self.scales, _U8, "scales", dev), self.form, 0, self.num_pages


class KV8Cache:
    """An 8-bit KV cache (layout: ``kv8_store`` in blockscore.h): ``codes``
    uint8 (or float8_e4m3fn) [slots, kv_heads, 2, head_dim] and ``scales``
    float32 [slots / 64, kv_heads, 2], contiguous, ``slots`` a multiple of 64.

    Its rows share a page's scale, so ``kv8_store`` asks more of its caller than
    ``kv4_store``: the rows of one page lie within 64 consecutive rows of a call, and
    a page's first slot is written before its others."""

    form = 8  # BS_KV_8

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dim() != 4 or codes.shape[2] != 2 or codes.shape[0] % PAGE_TOKENS:
            raise ValueError("codes must be [num_pages * 64, kv_heads, 2, head_dim]")
        self.codes, self.scales = codes, scales
        self.kv_heads, self.head_dim = int(codes.shape[1]), int(codes.shape[3])
        self.num_pages = int(codes.shape[0]) // PAGE_TOKENS
        if scales.shape != (self.num_pages, self.kv_heads, 2):
            raise ValueError("scales must be [num_pages, kv_heads, 2]")
        self.device = codes.device

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, head_dim: int, device) -> "KV8Cache":
        """Storage for ``num_pages`` pages (every slot reads back as zeros)."""
        n = int(num_pages)
        return cls(torch.zeros((n * PAGE_TOKENS, kv_heads, 2, head_dim), dtype=torch.uint8, device=device),
                   torch.full((n, kv_heads, 2), 2.0 ** -120, dtype=torch.float32, device=device))

    def _args(self, dtype, dev):
        return _ptr(self.codes, _CODES8, "codes", dev), _ptr(self.scales, _F32, "scales", dev), self.form, 0, self.num_pages


class KV16Cache:
    """K and V pools of the queries' 16-bit type: [slots, kv_heads, head_dim]
    each, ``slots`` a multiple of 64, both with the same stride from a slot to
    the next (views of one interleaved pool are fine)."""

    form = 0  # BS_KV_16

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if k.dim() != 3 or k.shape != v.shape or k.shape[0] % PAGE_TOKENS:
            raise ValueError("k and v must both be [num_pages * 64, kv_heads, head_dim]")
        if k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must have the same strides and dtype")
        self.k, self.v = k, v
        self.kv_heads, self.head_dim = int(k.shape[1]), int(k.shape[2])
        self.num_pages = int(k.shape[0]) // PAGE_TOKENS
        self.device = k.device

    def _args(self, dtype, dev):
        return (_rows_ptr(self.k, (dtype,), "k pool", dev), _rows_ptr(self.v, (dtype,), "v pool", dev), self.form,
                int(self.k.stride(0)), self.num_pages)


def _rows_ptr(t: torch.Tensor, dtypes, name: str, device):
    """Pointer of a [rows, heads, dim] tensor whose rows may lie apart."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dim() != 3 or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name} must be [rows, heads, dim] with contiguous rows")
    return C.c_void_p(t.data_ptr())


def _ld(t: torch.Tensor) -> int:
    """Elements from a row to the next (a lone row's stride means nothing)."""
    return int(t.stride(0)) if t.shape[0] > 1 else int(t.shape[1] * t.shape[2])


def _size(n) -> int:
    """A size for an int32 argument (which would wrap a larger one)."""
    if n > 2**31 - 1:
        raise ValueError(f"a size of {n} is more than 2^31 - 1")
    return int(n)


def _kv_store_args(k, v, slots, cache, kind):
    """Checked argument tuple of a ``kv4_store`` or ``kv8_store`` call (all but the stream)."""
    dev = cache.device
    if not isinstance(cache, kind):
        raise TypeError(f"cache must be a {kind.__name__}")
    if k.dim() != 3 or k.shape != v.shape or k.shape[1:] != (cache.kv_heads, cache.head_dim) or k.dtype != v.dtype:
        raise ValueError("k and v must both be [num_tok, kv_heads, head_dim] of one dtype")
    if slots.numel() != k.shape[0]:
        raise ValueError("slots must hold num_tok entries")
    codes, scales, _, _, num_pages = cache._args(None, dev)
    return (_rows_ptr(k, tuple(_DTYPES), "k", dev), _rows_ptr(v, tuple(_DTYPES), "v", dev), _DTYPES[k.dtype], _ld(k),
            _ld(v), _ptr(slots, _I32, "slots", dev), _size(k.shape[0]), cache.kv_heads, cache.head_dim, codes, scales,
            num_pages)


def kv4_store(k, v, slots, cache: KV4Cache, stream=None):
    """Quantise new K/V rows into the 4-bit cache.  See ``kv4_store`` in blockscore.h."""
    PreparedCall("kv4_store", _kv_store_args(k, v, slots, cache, KV4Cache), cache.device, once=True)(stream)


def kv8_store(k, v, slots, cache: KV8Cache, stream=None):
    """Quantise new K/V rows into the 8-bit cache.  The rows of one page (64 slots)
    must lie within 64 consecutive rows of the call, as ``pages_extend`` lists them:
    tokens ordered by step and then by request, say, are not written whole, which
    ``kv4_store`` would do.  A row for a page's first slot begins the page anew.  See
    ``kv8_store`` in blockscore.h."""
    PreparedCall("kv8_store", _kv_store_args(k, v, slots, cache, KV8Cache), cache.device, once=True)(stream)


def _kv_load_args(cache, slots, k, v, kind):
    """Checked argument tuple of a ``kv4_load`` or ``kv8_load`` call (all but the stream)."""
    dev = cache.device
    if not isinstance(cache, kind):
        raise TypeError(f"cache must be a {kind.__name__}")
    if k.dim() != 3 or k.shape != v.shape or k.shape[1:] != (cache.kv_heads, cache.head_dim) or k.dtype != v.dtype:
        raise ValueError("k and v must both be [num_slots, kv_heads, head_dim] of one dtype")
    if slots.numel() != k.shape[0]:
        raise ValueError("slots must hold one entry per row of k")
    codes, scales, _, _, num_pages = cache._args(None, dev)
    return (codes, scales, num_pages, _ptr(slots, _I32, "slots", dev), _size(k.shape[0]), cache.kv_heads,
            cache.head_dim, _rows_ptr(k, tuple(_DTYPES), "k", dev), _rows_ptr(v, tuple(_DTYPES), "v", dev),
            _DTYPES[k.dtype], _ld(k), _ld(v))


def kv4_load(cache: KV4Cache, slots, k, v, stream=None):
    """Read rows of the 4-bit cache back.  See ``kv4_load`` in blockscore.h."""
    PreparedCall("kv4_load", _kv_load_args(cache, slots, k, v, KV4Cache), cache.device, once=True)(stream)


def kv8_load(cache: KV8Cache, slots, k, v, stream=None):
    """Read rows of the 8-bit cache back.  See ``kv8_load`` in blockscore.h."""
    PreparedCall("kv8_load", _kv_load_args(cache, slots, k, v, KV8Cache), cache.device, once=True)(stream)


class Idx4Cache:
    """Index keys in 4 bits (layout: ``idx4_store`` in blockscore.h): ``codes``
    uint8 [keys, 64] and ``scales`` uint8 [keys, 4], contiguous, ``keys`` a
    multiple of 64 / c."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, c: int):
        if int(c) not in (1, 4):
            raise ValueError("c must be 1 or 4")
        if codes.dim() != 2 or codes.shape[1] != DIM // 2 or codes.shape[0] % (PAGE_TOKENS // int(c)):
            raise ValueError("codes must be [num_pages * (64 / c), 64]")
        if scales.shape != (codes.shape[0], DIM // 32):
            raise ValueError("scales must be [num_pages * (64 / c), 4]")
        self.codes, self.scales, self.c = codes, scales, int(c)
        self.num_keys = int(codes.shape[0])
        self.num_pages = self.num_keys // (PAGE_TOKENS // self.c)
        self.device = codes.device

    @classmethod
    def empty(cls, num_pages: int, c: int, device) -> "Idx4Cache":
        """Storage for ``num_pages`` pages (every key reads back as zeros)."""
        n = int(num_pages) * (PAGE_TOKENS // int(c))
        return cls(torch.zeros((n, DIM // 2), dtype=torch.uint8, device=device),
                   torch.full((n, DIM // 32), 127, dtype=torch.uint8, device=device), c)

    def _ptrs(self, dev):
        return _ptr(self.codes, _U8, "codes", dev), _ptr(self.scales, _U8, "scales", dev)


def _keys_ptr(t: torch.Tensor, name: str, rows: int, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != DIM:
        raise ValueError(f"{name} must be [rows, 128], one row per slot")
    return _rows_ptr(t.unsqueeze(1), tuple(_DTYPES), name, dev), _DTYPES[t.dtype], _ld(t.unsqueeze(1))


def _idx4_cache(cache):
    if not isinstance(cache, Idx4Cache):
        raise TypeError("cache must be an Idx4Cache")
    return cache.device


def _idx4_store_args(keys, slots, cache):
    """Checked argument tuple of an ``idx4_store`` call (all but the stream)."""
    dev = _idx4_cache(cache)
    n = _size(slots.numel())
    return (*_keys_ptr(keys, "keys", n, dev), _ptr(slots, _I32, "slots", dev), n, *cache._ptrs(dev),
            _size(cache.num_keys))


def idx4_store(keys, slots, cache: Idx4Cache, stream=None):
    """Quantise index keys into the 4-bit cache.  See ``idx4_store`` in blockscore.h."""
    PreparedCall("idx4_store", _idx4_store_args(keys, slots, cache), cache.device, once=True)(stream)


def _idx4_load_args(cache, slots, keys):
    """Checked argument tuple of an ``idx4_load`` call (all but the stream)."""
    dev = _idx4_cache(cache)
    n = _size(slots.numel())
    return (*cache._ptrs(dev), _size(cache.num_keys), _ptr(slots, _I32, "slots", dev), n,
            *_keys_ptr(keys, "keys", n, dev))


def idx4_load(cache: Idx4Cache, slots, keys, stream=None):
    """Read 4-bit index keys back.  See ``idx4_load`` in blockscore.h."""
    PreparedCall("idx4_load", _idx4_load_args(cache, slots, keys), cache.device, once=True)(stream)


def _idx4_compress_args(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok, rotary_dim, sections, theta, ring, ring_pos,
                        page_table, cache):
    """Checked argument tuple of an ``idx4_compress_store_ring`` call (all but the stream)."""
    _idx4_cache(cache)
    if cache.c != 4:
        raise ValueError("compressed keys go to a cache of c = 4")
    return (*_compress_head(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok, rotary_dim, sections, theta, ring,
                            ring_pos, page_table), *cache._ptrs(k_raw.device), cache.num_pages)


def idx4_compress_store(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok, rotary_dim, sections, theta, ring, ring_pos,
                        page_table, cache: Idx4Cache, stream=None):
    """Compress new raw index keys into the 4-bit c = 4 keys (and update the
    rings, which are ``idx_compress_store``'s).  See ``idx4_compress_store`` in
    blockscore.h."""
    PreparedCall("idx4_compress_store_ring", _idx4_compress_args(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok,
                                                                 rotary_dim, sections, theta, ring, ring_pos,
                                                                 page_table, cache), k_raw.device, once=True)(stream)


def _idx4_score_args(q, cache, page_table, req_row_ptr, row_pos, max_vis, scores, row_len=None):
    """Checked argument tuple of an ``idx4_score`` call (all but the stream)."""
    _idx4_cache(cache)
    a = _score_args(q, None, cache.num_pages, page_table, req_row_ptr, row_pos, cache.c, max_vis, scores, row_len)
    return (a[0], *cache._ptrs(q.device), *a[2:])


def idx4_score(q, cache: Idx4Cache, page_table, req_row_ptr, row_pos, max_vis, scores, row_len=None, stream=None):
    """Scores over 4-bit index keys, any number of rows a request.  See ``idx4_score`` in blockscore.h."""
    PreparedCall("idx4_score", _idx4_score_args(q, cache, page_table, req_row_ptr, row_pos, max_vis, scores, row_len),
                 q.device, once=True)(stream)


class PagePool:
    """The free pages of a cache: ``ring`` int32 [size], their ids, and
    ``state`` int32 [4], head, count, what the last ``pages_extend`` lacked, 0
    (``pages_extend`` in blockscore.h; a state made by hand needs the 0, one that is
    only written, a ``pool_out``, may hold anything)."""

    def __init__(self, ring: torch.Tensor, state: torch.Tensor):
        if ring.dim() != 1 or state.shape != (4,):
            raise ValueError("ring must be [size] and state [4]")
        self.ring, self.state = ring, state

    @classmethod
    def full(cls, num_pages: int, device) -> "PagePool":
        """All of ``num_pages`` pages, free."""
        n = _size(num_pages)
        return cls(torch.arange(n, dtype=torch.int32, device=device),
                   torch.tensor([0, n, 0, 0], dtype=torch.int32, device=device))


def _pages_args(pool, kv_len, held, change, name, page_table, kv_len_out, held_out, pool_out):
    if not isinstance(pool, PagePool) or not (pool_out is None or isinstance(pool_out, PagePool)):
        raise TypeError("pool and pool_out must be PagePools")
    dev = pool.ring.device
    B = kv_len.numel()
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [num_req, pt_stride]")
    outs = [x if y is None else y for x, y in ((kv_len, kv_len_out), (held, held_out), (pool, pool_out))]
    if any(x.numel() != B for x in (held, change, *outs[:2])):
        raise ValueError(f"held, {name}, kv_len_out and held_out must hold num_req entries")
    if outs[2].ring.data_ptr() != pool.ring.data_ptr():
        raise ValueError("pool_out must be of the same ring")
    return (_ptr(kv_len, _I32, "kv_len", dev), _ptr(held, _I32, "held", dev), _ptr(change, _I32, name, dev), _size(B),
            _ptr(page_table, _I32, "page_table", dev), _size(page_table.shape[1]), _ptr(pool.ring, _I32, "ring", dev),
            _size(pool.ring.numel()), _ptr(pool.state, _I32, "state", dev), _ptr(outs[0], _I32, "kv_len_out", dev),
            _ptr(outs[1], _I32, "held_out", dev), _ptr(outs[2].state, _I32, "state", dev))


def _pages_extend_args(pool, kv_len, held, new_len, page_table, req_row_ptr, row_pos, slots, tok_start=None,
                       kv_len_out=None, held_out=None, pool_out=None):
    """Checked argument tuple of a ``pages_extend`` call (all but the stream)."""
    a = _pages_args(pool, kv_len, held, new_len, "new_len", page_table, kv_len_out, held_out, pool_out)
    dev = pool.ring.device
    if req_row_ptr.numel() != kv_len.numel() + 1 or slots.numel() != row_pos.numel():
        raise ValueError("req_row_ptr must hold num_req + 1 entries, row_pos and slots num_rows each")
    if tok_start is not None and tok_start.numel() != kv_len.numel():
        raise ValueError("tok_start must hold num_req entries")
    return (*a, _ptr(req_row_ptr, _I32, "req_row_ptr", dev), _ptr(tok_start, _I32, "tok_start", dev), _ptr(row_pos, _I32, "row_pos", dev),
            _ptr(slots, _I32, "slots", dev), _size(row_pos.numel()))


def pages_extend(pool: PagePool, kv_len, held, new_len, page_table, req_row_ptr, row_pos, slots, tok_start=None,
                 kv_len_out=None, held_out=None, pool_out=None, stream=None):
    """Append new tokens to a batch: their pages, positions and slots.  The
    state is updated in place unless told otherwise (``pool_out``: a PagePool of
    the same ring).  See ``pages_extend`` in blockscore.h."""
    PreparedCall("pages_extend", _pages_extend_args(pool, kv_len, held, new_len, page_table, req_row_ptr, row_pos,
                                                    slots, tok_start, kv_len_out, held_out, pool_out),
                 pool.ring.device, once=True)(stream)


def _pages_release_args(pool, kv_len, held, keep_len, page_table, kv_len_out=None, held_out=None, pool_out=None):
    """Checked argument tuple of a ``pages_release`` call (all but the stream)."""
    return _pages_args(pool, kv_len, held, keep_len, "keep_len", page_table, kv_len_out, held_out, pool_out)


def pages_release(pool: PagePool, kv_len, held, keep_len, page_table, kv_len_out=None, held_out=None, pool_out=None,
                  stream=None):
    """Cut requests back and return their pages.  See ``pages_release`` in blockscore.h."""
    PreparedCall("pages_release", _pages_release_args(pool, kv_len, held, keep_len, page_table, kv_len_out, held_out,
                                                      pool_out), pool.ring.device, once=True)(stream)


def attn_workspace(device) -> torch.Tensor:
    """A zero-filled workspace that serves every ``attn_slots`` and
    ``attn_window`` call on one stream: the current one, which clears it (to be
    done outside a graph that is being captured)."""
    return torch.zeros(ATTN_WORKSPACE_BYTES, dtype=torch.uint8, device=device)


def _attn_common(q, cache, out, scale, lse, workspace):
    dev = q.device
    if q.dim() != 3 or out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("q and out must both be [num_rows, q_heads, head_dim] of one dtype")
    if q.shape[2] != cache.head_dim or q.shape[1] % cache.kv_heads:
        raise ValueError("q does not fit the cache's heads")
    if lse is not None and lse.shape != q.shape[:2]:
        raise ValueError("lse must be [num_rows, q_heads]")
    half = (torch.bfloat16, torch.float16)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    head = (_rows_ptr(q, half, "q", dev), _DTYPES[q.dtype], _ld(q), _size(q.shape[0]), int(q.shape[1]), cache.kv_heads,
            cache.head_dim, *cache._args(q.dtype, dev))
    tail = (float(scale) if scale is not None else 1.0 / math.sqrt(cache.head_dim), _rows_ptr(out, half, "out", dev),
            _ld(out), _ptr(lse, _F32, "lse", dev), _ptr(workspace, _U8, "workspace", dev), ws_bytes)
    return head, tail


def _attn_slots_args(q, cache, slots, out, count=None, scale=None, lse=None, workspace=None):
    """Checked argument tuple of an ``attn_slots`` call (all but the stream)."""
    dev = q.device
    head, tail = _attn_common(q, cache, out, scale, lse, workspace)
    if slots.dim() != 2 or slots.shape[0] != q.shape[0]:
        raise ValueError("slots must be [num_rows, ld_slots]")
    if count is not None and count.numel() != q.shape[0]:
        raise ValueError("count must hold num_rows entries")
    return (*head, _ptr(slots, _I32, "slots", dev), _size(slots.shape[1]), _ptr(count, _I32, "count", dev), *tail)


def attn_slots(q, cache, slots, out, count=None, scale=None, lse=None, workspace=None, stream=None):
    """Attention of each row over its slots (``scale`` defaults to
    1/sqrt(head_dim)).  See ``attn_slots`` in blockscore.h."""
    PreparedCall("attn_slots", _attn_slots_args(q, cache, slots, out, count, scale, lse, workspace), q.device,
                 once=True)(stream)


def _int32(x) -> int:
    """``x`` for an int32 argument that bounds positions or rows, which are
    int32 themselves: a larger bound (no window: 1 << 40, say) means the same as
    the largest."""
    return max(min(int(x), 2**31 - 1), -1)


def _attn_window_args(q, cache, page_table, req_row_ptr, row_pos, max_rows, window, sinks, out, scale=None, lse=None,
                      workspace=None):
    """Checked argument tuple of an ``attn_window`` call (all but the stream)."""
    dev = q.device
    head, tail = _attn_common(q, cache, out, scale, lse, workspace)
    B = int(req_row_ptr.shape[0]) - 1
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [num_req, pt_stride]")
    if row_pos.numel() != q.shape[0]:
        raise ValueError("row_pos must hold num_rows entries")
    return (*head, _ptr(page_table, _I32, "page_table", dev), _size(page_table.shape[1]),
            _ptr(req_row_ptr, _I32, "req_row_ptr", dev), _size(B), _ptr(row_pos, _I32, "row_pos", dev), *map(_int32, (
                max_rows, window, sinks)), *tail)


def attn_window(q, cache, page_table, req_row_ptr, row_pos, max_rows, window, sinks, out, scale=None, lse=None,
                workspace=None, stream=None):
    """Attention over a sliding window and the first ``sinks`` tokens
    (``scale`` defaults to 1/sqrt(head_dim)).  See ``attn_window`` in
    blockscore.h."""
    PreparedCall("attn_window", _attn_window_args(q, cache, page_table, req_row_ptr, row_pos, max_rows, window, sinks,
                                                  out, scale, lse, workspace), q.device, once=True)(stream)


class PreparedCall:
    """One C call with its arguments checked and marshalled once (the tensors
    behind the pointers must outlive it); ``__call__`` adds the stream and
    checks the status.  For loops that issue the same call many times."""

    def __init__(self, fn: str, args: tuple, device, once: bool = False):
        self.fn = fn
        self.args = args
        self.device = device
        self._f = getattr(lib(), fn)
        # Arguments as instances of their declared C types, so that a call
        # converts nothing but the stream (worth it for more than one call).
        self._args = args if once else tuple(a if isinstance(a, t) else t(a) for a, t in zip(args, self._f.argtypes))

    def __call__(self, stream=None):
        # The current stream and device are asked for by their index: about
        # 1 us less per call than through torch's Stream objects.
        index = self.device.index
        if index == torch._C._cuda_getDevice():
            s = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
            st = self._f(*self._args, s)
        else:  # a launch goes to the current device, and the tensors live on another
            with torch.cuda.device(self.device):
                st = self._f(*self._args, _stream(stream, self.device))
        if st != 0:
            _check(st, self.fn)

    def bind(self, stream=None) -> "BoundCall":
        """The same call with the stream resolved now (default: the current
        stream): each call is then one C call with nothing looked up (the
        tensors' device must be the current one)."""
        return BoundCall(self, _stream(stream, self.device))


class BoundCall:
    """A PreparedCall with its stream fixed; ``__call__`` takes no arguments."""

    __slots__ = ("fn", "_f", "_args")

    def __init__(self, prepared: PreparedCall, stream_ptr):
        self.fn = prepared.fn
        self._f = prepared._f
        self._args = (*prepared._args, stream_ptr)

    def __call__(self):
        st = self._f(*self._args)
        if st != 0:
            _check(st, self.fn)


def prepare_score(fn: str, q, kcache, num_pages, page_table, req_row_ptr, row_pos, c, max_vis, scores,
                  row_len=None) -> PreparedCall:
    """``idx_score_decode`` or ``idx_score_prefill`` with fixed arguments."""
    if fn not in ("idx_score_decode", "idx_score_prefill"):
        raise ValueError("fn must be idx_score_decode or idx_score_prefill")
    return PreparedCall(fn, _score_args(q, kcache, num_pages, page_table, req_row_ptr, row_pos, c, max_vis,
                                        scores, row_len), q.device)


def prepare_topk(scores, row_len, max_len, k, sel, sel_count, workspace=None) -> PreparedCall:
    """``topk_select_rows`` with fixed arguments."""
    return PreparedCall("topk_select_rows", _topk_args(scores, row_len, max_len, k, sel, sel_count, workspace),
                        scores.device)


def prepare_expand_shared(sel, sel_count, k, req_row_ptr, row_pos, row_pos_now, c, max_advance, page_table,
                          out_slots, out_count, out_pos=None) -> PreparedCall:
    """``idx_expand_translate_shared`` with fixed arguments."""
    return PreparedCall("idx_expand_translate_shared",
                        _expand_shared_args(sel, sel_count, k, req_row_ptr, row_pos, row_pos_now, c, max_advance,
                                            page_table, out_slots, out_count, out_pos), sel.device)


def prepare_select_translate(scores, row_len, max_len, k, req_row_ptr, row_pos, c, page_table, sel, sel_count,
                             out_slots, out_count, out_pos=None, workspace=None) -> PreparedCall:
    """``idx_select_translate`` with fixed arguments."""
    return PreparedCall("idx_select_translate",
                        _select_translate_args(scores, row_len, max_len, k, req_row_ptr, row_pos, c, page_table,
                                               sel, sel_count, out_slots, out_count, out_pos, workspace),
                        scores.device)


def prepare_plan(row_len, max_len, plan) -> PreparedCall:
    """``topk_plan_rows`` with fixed arguments."""
    return PreparedCall("topk_plan_rows", _plan_args(row_len, max_len, plan), row_len.device)


def prepare_select_translate_planned(scores, max_len, k, req_row_ptr, row_pos, c, page_table, sel, sel_count,
                                     out_slots, out_count, plan, out_pos=None, workspace=None) -> PreparedCall:
    """``idx_select_translate_planned`` with fixed arguments."""
    return PreparedCall("idx_select_translate_planned",
                        _select_translate_planned_args(scores, max_len, k, req_row_ptr, row_pos, c, page_table, sel,
                                                       sel_count, out_slots, out_count, plan, out_pos, workspace),
                        scores.device)


__all__ = [
    "idx_score_decode", "idx_score_prefill", "topk_workspace_bytes", "topk_workspace",
    "topk_select_rows", "idx_expand_translate", "idx_expand_translate_shared", "idx_select_translate",
    "idx_select_translate_noalloc", "NOALLOC_SCRATCH_BYTES", "idx_compress_store", "status_string", "BlockScoreError",
    "lib", "PreparedCall", "BoundCall", "prepare_score", "prepare_topk", "prepare_select_translate", "prepare_expand_shared",
    "prepare_compress_store", "topk_plan_bytes", "topk_planned_workspace_bytes", "topk_plan",
    "topk_planned_workspace", "topk_plan_rows", "idx_select_translate_planned", "prepare_plan",
    "prepare_select_translate_planned", "KV4Cache", "KV16Cache", "kv4_store", "kv4_load", "attn_workspace",
    "ATTN_WORKSPACE_BYTES", "attn_slots", "attn_window", "prepare_kv4_store", "prepare_kv4_load",
    "prepare_attn_slots", "prepare_attn_window", "KV8Cache", "kv8_store", "kv8_load", "prepare_kv8_store",
    "prepare_kv8_load", "Idx4Cache", "idx4_store", "idx4_load", "idx4_compress_store", "idx4_score",
    "prepare_idx4_store", "prepare_idx4_load", "prepare_idx4_compress_store", "prepare_idx4_score", "PagePool",
    "pages_extend", "pages_release", "prepare_pages_extend", "prepare_pages_release",
]


def prepare_compress_store(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok, rotary_dim, sections, theta, ring,
                           ring_pos, page_table, kcache, num_pages) -> PreparedCall:
    """``idx_compress_store`` with fixed arguments."""
    return PreparedCall("idx_compress_store_ring",
                        _compress_args(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok, rotary_dim, sections,
                                       theta, ring, ring_pos, page_table, kcache, num_pages), k_raw.device)


def prepare_kv4_store(k, v, slots, cache: KV4Cache) -> PreparedCall:
    """``kv4_store`` with fixed arguments."""
    return PreparedCall("kv4_store", _kv_store_args(k, v, slots, cache, KV4Cache), cache.device)


def prepare_kv4_load(cache: KV4Cache, slots, k, v) -> PreparedCall:
    """``kv4_load`` with fixed arguments."""
    return PreparedCall("kv4_load", _kv_load_args(cache, slots, k, v, KV4Cache), cache.device)


def prepare_kv8_store(k, v, slots, cache: KV8Cache) -> PreparedCall:
    """``kv8_store`` with fixed arguments."""
    return PreparedCall("kv8_store", _kv_store_args(k, v, slots, cache, KV8Cache), cache.device)


def prepare_kv8_load(cache: KV8Cache, slots, k, v) -> PreparedCall:
    """``kv8_load`` with fixed arguments."""
    return PreparedCall("kv8_load", _kv_load_args(cache, slots, k, v, KV8Cache), cache.device)


def prepare_idx4_store(keys, slots, cache: Idx4Cache) -> PreparedCall:
    """``idx4_store`` with fixed arguments."""
    return PreparedCall("idx4_store", _idx4_store_args(keys, slots, cache), cache.device)


def prepare_idx4_load(cache: Idx4Cache, slots, keys) -> PreparedCall:
    """``idx4_load`` with fixed arguments."""
    return PreparedCall("idx4_load", _idx4_load_args(cache, slots, keys), cache.device)


def prepare_idx4_compress_store(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok, rotary_dim, sections, theta, ring,
                                ring_pos, page_table, cache: Idx4Cache) -> PreparedCall:
    """``idx4_compress_store`` with fixed arguments."""
    return PreparedCall("idx4_compress_store_ring", _idx4_compress_args(k_raw, req_tok_ptr, tok_start, mrope_pos, max_tok,
                                                                   rotary_dim, sections, theta, ring, ring_pos,
                                                                   page_table, cache), k_raw.device)


def prepare_idx4_score(q, cache: Idx4Cache, page_table, req_row_ptr, row_pos, max_vis, scores,
                       row_len=None) -> PreparedCall:
    """``idx4_score`` with fixed arguments."""
    return PreparedCall("idx4_score", _idx4_score_args(q, cache, page_table, req_row_ptr, row_pos, max_vis, scores,
                                                       row_len), q.device)


def prepare_pages_extend(pool: PagePool, kv_len, held, new_len, page_table, req_row_ptr, row_pos, slots,
                         tok_start=None, kv_len_out=None, held_out=None, pool_out=None) -> PreparedCall:
    """``pages_extend`` with fixed arguments."""
    return PreparedCall("pages_extend", _pages_extend_args(pool, kv_len, held, new_len, page_table, req_row_ptr,
                                                           row_pos, slots, tok_start, kv_len_out, held_out,
                                                           pool_out), pool.ring.device)


def prepare_pages_release(pool: PagePool, kv_len, held, keep_len, page_table, kv_len_out=None, held_out=None,
                          pool_out=None) -> PreparedCall:
    """``pages_release`` with fixed arguments."""
    return PreparedCall("pages_release", _pages_release_args(pool, kv_len, held, keep_len, page_table, kv_len_out,
                                                             held_out, pool_out), pool.ring.device)


def prepare_attn_slots(q, cache, slots, out, count=None, scale=None, lse=None, workspace=None) -> PreparedCall:
    """``attn_slots`` with fixed arguments."""
    return PreparedCall("attn_slots", _attn_slots_args(q, cache, slots, out, count, scale, lse, workspace), q.device)


def prepare_attn_window(q, cache, page_table, req_row_ptr, row_pos, max_rows, window, sinks, out, scale=None, lse=None,
                        workspace=None) -> PreparedCall:
    """``attn_window`` with fixed arguments."""
    return PreparedCall("attn_window", _attn_window_args(q, cache, page_table, req_row_ptr, row_pos, max_rows, window,
                                                         sinks, out, scale, lse, workspace), q.device)
