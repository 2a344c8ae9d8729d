"""The paged key-value cache: page tables of a step (``thd_paged_tables``) and
attention of one new token per request over its pages (``thd_paged_decode``), as
declared in include/thd_attn.h. ``norm_rope.thd_qk_norm_rope_append`` fills the cache.

The functions that take a plan only marshal arguments, like ``thd_attn_fwd``; the
one-call functions check shapes, make the plan (cached) and allocate what is not given.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import binding as _b


class ThdPagedTablesDesc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("table_stride", ctypes.c_int64),
        ("cap_rows", ctypes.c_int32),
        ("cap_free", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
    ]


class ThdPagedDecodeDesc(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("batch", ctypes.c_int32),
        ("h_q", ctypes.c_int32),
        ("h_kv", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("table_stride", ctypes.c_int64),
        ("stride_tok", ctypes.c_int64 * 4),
        ("stride_head", ctypes.c_int64 * 4),
        ("stride_page", ctypes.c_int64 * 4),
        ("bytes", ctypes.c_int64 * 4),
        ("stats_layout", ctypes.c_int),
        ("softmax_scale", ctypes.c_float),
        ("kernel", ctypes.c_int),
        ("flags", ctypes.c_uint32),
    ]


def _check_table(block_table, batch: int) -> None:
    if block_table.dim() != 2 or block_table.dtype != torch.int32 or block_table.shape[0] != batch or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1) or \
            (batch > 1 and block_table.stride(0) < block_table.shape[1]):
        raise ValueError("block_table must be int32 [batch, max_pages] with a contiguous last dim")


def _table_stride(block_table) -> int:
    # the stride of a table of one row (or none) says nothing
    return max(block_table.stride(0), block_table.shape[1])


# ------------------------------------------------------------------------------- page tables
def paged_tables_plan(batch: int, page_size: int, num_pages: int, max_pages: int, table_stride: int, cap_rows: int,
                      cap_free: int) -> _b.ThdAttnPlan:
    """Plan of the page tables of a step (see ``thd_paged_tables_desc_t``)."""
    d = ThdPagedTablesDesc()
    d.batch, d.page_size, d.num_pages, d.max_pages = batch, page_size, num_pages, max_pages
    d.table_stride, d.cap_rows, d.cap_free, d.flags = table_stride, cap_rows, cap_free, 0
    return _b.make_plan("thd_paged_tables_plan", d)


def thd_paged_tables(plan, seq_lens, cu_new, free_pages, free_span, block_table, slot_map, positions, seq_lens_out,
                     free_begin_out, workspace, stream=None) -> None:
    """Enqueue the page tables of a step (see ``thd_paged_tables`` in include/thd_attn.h);
    every tensor but the workspace is int32 on the device."""
    _b._enqueue("thd_paged_tables", plan, seq_lens, (seq_lens, cu_new, free_pages, free_span, block_table, slot_map,
                                                     positions, seq_lens_out, free_begin_out, workspace), stream)


def thd_paged_extend(seq_lens, cu_new, free_pages, free_span, block_table, *, page_size: int, num_pages: int,
                     rows: int | None = None, slot_map=None, positions=None, seq_lens_out=None, free_begin_out=None,
                     workspace=None, stream=None):
    """One-call page tables: pages for the new tokens ``cu_new`` (int32 [B+1]) of requests
    that hold ``seq_lens`` (int32 [B]) tokens, entered into ``block_table`` (int32
    [B, max_pages], in place), from ``free_pages[free_span[0]:free_span[1]]``. ``rows`` is the
    capacity of the step's packed rows (or give ``slot_map`` / ``positions``). Returns
    ``(slot_map, positions, seq_lens_out, free_begin_out)``."""
    batch = seq_lens.numel()
    if rows is None:
        given = slot_map if slot_map is not None else positions
        if given is None:
            raise ValueError("give rows, slot_map or positions")
        rows = given.numel()
    _check_table(block_table, batch)
    for name, t, shape in (("seq_lens", seq_lens, (batch,)), ("cu_new", cu_new, (batch + 1,)),
                           ("free_pages", free_pages, (free_pages.numel(),)), ("free_span", free_span, (2,)),
                           ("slot_map", slot_map, (rows,)), ("positions", positions, (rows,)),
                           ("seq_lens_out", seq_lens_out, (batch,)), ("free_begin_out", free_begin_out, (1,))):
        if t is not None:
            _b._check_ints(name, t, shape)
    _b._check_devices(seq_lens, cu_new, free_pages, free_span, block_table, slot_map, positions, seq_lens_out,
                      free_begin_out)
    with _b._allocating_on(seq_lens, stream):
        new = lambda t, n: torch.empty(n, dtype=torch.int32, device=seq_lens.device) if t is None else t  # noqa: E731
        slot_map, positions = new(slot_map, rows), new(positions, rows)
        seq_lens_out, free_begin_out = new(seq_lens_out, batch), new(free_begin_out, 1)
        key = ("paged_tables", batch, page_size, num_pages, block_table.shape[1], _table_stride(block_table), rows,
               free_pages.numel())
        plan = _b._cached_plan(key, lambda: paged_tables_plan(*key[1:]))
        if workspace is None:
            workspace = _b.alloc_workspace(plan, seq_lens.device)
        thd_paged_tables(plan, seq_lens, cu_new, free_pages, free_span, block_table, slot_map, positions, seq_lens_out,
                         free_begin_out, workspace, stream)
    return slot_map, positions, seq_lens_out, free_begin_out


# ---------------------------------------------------------------------- one-token attention
def paged_decode_plan(desc: ThdPagedDecodeDesc) -> _b.ThdAttnPlan:
    return _b.make_plan("thd_paged_decode_plan", desc)


def paged_decode_plan_for_tensors(q, k_cache, v_cache, o, block_table, *, stats_layout: int = _b.STATS_TOKEN_MAJOR,
                                  softmax_scale=None, kernel: int = _b.KERNEL_AUTO) -> _b.ThdAttnPlan:
    """Plan from Q and O [batch, h_q, d], the caches as [pages, page_size, h_kv, d] views of
    any strides (a [pages, h_kv, page_size, d] buffer is passed transposed) and the block
    table int32 [batch, max_pages]; last dims contiguous."""
    if q.dim() != 3 or o.shape != q.shape or k_cache.dim() != 4 or v_cache.shape != k_cache.shape or \
            k_cache.shape[3] != q.shape[2]:
        raise ValueError("Q and O must be [batch, h_q, d], the caches [pages, page_size, h_kv, d]")
    for t in (q, k_cache, v_cache, o):
        if t.stride(-1) != 1:
            raise ValueError("Q, O and the caches must have a contiguous last dim")
        if t.dtype != q.dtype or t.dtype not in _b._DTYPE_CODE:
            raise ValueError("Q, O and the caches must share one storage type: bfloat16, float16 or float32")
    _check_table(block_table, q.shape[0])
    d = ThdPagedDecodeDesc()
    d.dtype = _b._DTYPE_CODE[q.dtype]
    d.batch, d.h_q, d.d = q.shape
    d.num_pages, d.page_size, d.h_kv = k_cache.shape[:3]
    d.max_pages, d.table_stride = block_table.shape[1], _table_stride(block_table)
    for i, t in enumerate((q, k_cache, v_cache, o)):
        d.stride_tok[i], d.stride_head[i] = t.stride(-3), t.stride(-2)
        d.stride_page[i] = t.stride(0) if t.dim() == 4 else 0
        d.bytes[i] = _b._view_bytes(t)
    d.stats_layout = int(stats_layout)
    d.softmax_scale = math.nan if softmax_scale is None else float(softmax_scale)
    d.kernel, d.flags = int(kernel), 0
    return paged_decode_plan(d)


def thd_paged_decode(plan, q, k_cache, v_cache, block_table, seq_lens, window_left, o, stats, workspace,
                     stream=None) -> None:
    """Enqueue one-token attention (see ``thd_paged_decode`` in include/thd_attn.h);
    ``window_left`` and ``stats`` may be None."""
    _b._enqueue("thd_paged_decode", plan, q, (q, k_cache, v_cache, block_table, seq_lens, window_left, o, stats,
                                              workspace), stream)


def thd_paged_attention(q, k_cache, v_cache, block_table, seq_lens, *, window_left=None, o=None, stats=None,
                        stats_layout: int = _b.STATS_TOKEN_MAJOR, softmax_scale=None, kernel: int = _b.KERNEL_AUTO,
                        workspace=None, stream=None):
    """One-call attention of one new token per request: Q [batch, h_q, d] against the
    ``seq_lens[b]`` cached keys of each request (int32 [batch], the new token's own among
    them), whose pages ``block_table`` (int32 [batch, max_pages]) names. ``window_left``
    (int32 [batch], negative: none) bounds the keys from the left. For inference: no gradient
    flows through it. Returns ``(o, stats)``."""
    _b._check_ints("seq_lens", seq_lens, (q.shape[0],))
    if window_left is not None:
        _b._check_ints("window_left", window_left, (q.shape[0],))
    rows = q.shape[0] * q.shape[1]
    if stats is not None and (stats.dtype != torch.float32 or stats.numel() < rows or not stats.is_contiguous()):
        raise ValueError("stats must be contiguous float32 of batch * h_q entries")
    _b._check_devices(q, k_cache, v_cache, block_table, seq_lens, window_left, o, stats)
    with _b._allocating_on(q, stream):
        # a request of invalid length keeps its rows as they were: defined values, then
        if o is None:
            o = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        if stats is None:
            stats = torch.full((rows,), float("-inf"), dtype=torch.float32, device=q.device)
        key = ("paged_decode", tuple((t.dtype, tuple(t.shape), t.stride(), _b._view_bytes(t))
                                     for t in (q, k_cache, v_cache, o)),
               block_table.dtype, tuple(block_table.shape), block_table.stride(), stats_layout, softmax_scale, kernel)
        plan = _b._cached_plan(key, lambda: paged_decode_plan_for_tensors(
            q, k_cache, v_cache, o, block_table, stats_layout=stats_layout, softmax_scale=softmax_scale, kernel=kernel))
        if workspace is None:
            workspace = _b.alloc_workspace(plan, q.device)
        thd_paged_decode(plan, q, k_cache, v_cache, block_table, seq_lens, window_left, o, stats, workspace, stream)
    return o, stats
