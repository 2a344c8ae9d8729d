"""Checks of the norm-with-rotation, page-table and one-token-attention entry points
that need no GPU: exports, descriptors that are refused, calls that are refused before
anything is launched, and the one-call functions' argument checks."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

import ragged_varlen_attention_gb300 as rva
from ragged_varlen_attention_gb300 import binding as bd
from ragged_varlen_attention_gb300 import norm_rope as nr
from ragged_varlen_attention_gb300 import paged as pg

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "thd_attn.h")
P = 4096   # a non-null, aligned pointer that no refused call follows


@pytest.fixture(scope="module", autouse=True)
def lib():
    from ragged_varlen_attention_gb300 import build
    build.build()
    return bd.load_library()


def _plan(lib, entry, desc):
    h, ws = ctypes.c_void_p(), ctypes.c_size_t()
    st = getattr(lib, entry)(ctypes.byref(h), ctypes.byref(desc), ctypes.byref(ws))
    return st, (h if st == 0 else None), ws.value


def _set(desc, **kw):
    for name, v in kw.items():
        if hasattr(getattr(desc, name), "__len__"):
            for i, x in enumerate(v):
                getattr(desc, name)[i] = x
        else:
            setattr(desc, name, v)
    return desc


def _norm(**kw):
    base = dict(dtype=0, form=0, rows=10, h_q=4, h_kv=2, d=64, rot=32, interleaved=0, max_pos=100, eps=1e-6, page_size=4,
                num_pages=5, stride_tok=(256, 128, 128, 256, 128, 128), stride_head=(64,) * 6, stride_page=(512,) * 6,
                bytes=(0,) * 6, flags=0)
    base.update(kw)
    return _set(nr.ThdNormRopeDesc(), **base)


def _tables(**kw):
    base = dict(batch=3, page_size=4, num_pages=20, max_pages=6, table_stride=6, cap_rows=10, cap_free=9, flags=0)
    base.update(kw)
    return _set(pg.ThdPagedTablesDesc(), **base)


def _decode(**kw):
    base = dict(dtype=0, batch=3, h_q=4, h_kv=2, d=64, page_size=4, num_pages=20, max_pages=6, table_stride=6,
                stride_tok=(256, 128, 128, 256), stride_head=(64,) * 4, stride_page=(0, 512, 512, 0), bytes=(0,) * 4,
                stats_layout=0, softmax_scale=float("nan"), kernel=0, flags=0)
    base.update(kw)
    return _set(pg.ThdPagedDecodeDesc(), **base)


def test_every_declared_entry_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(thd_(?:qk_norm_rope|paged)_[a-z_]+)\s*\(", text))
    assert len(names) == 8
    for n in names:
        assert hasattr(lib, n) and n in bd._EXPORTS


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), 1), (dict(form=3), 1), (dict(rows=-1), 1), (dict(h_q=0), 1), (dict(h_kv=0), 1), (dict(d=0), 1),
    (dict(rot=3), 1), (dict(rot=66), 1), (dict(rot=-2), 1), (dict(max_pos=-1), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(flags=1), 1), (dict(stride_tok=(-1, 1, 1, 1, 1, 1)), 1),
    (dict(d=264, rot=0), 2), (dict(bytes=((9 * 256 + 3 * 64 + 64) * 2 - 2, 0, 0, 0, 0, 0)), 4),
    (dict(form=2, page_size=0), 1), (dict(form=2, num_pages=-1), 1),
    (dict(form=2, page_size=1 << 16, num_pages=1 << 15), 2),
    (dict(form=2, stride_page=(0, 0, 0, 0, -1, 0)), 1),
    (dict(form=2, bytes=(0, 0, 0, 0, 0, (4 * 512 + 3 * 128 + 64 + 64) * 2 - 2)), 4),
])
def test_norm_rope_descriptors_refused(lib, kw, code):
    assert _plan(lib, "thd_qk_norm_rope_plan", _norm(**kw))[0] == code


def test_norm_rope_exact_spans_accepted(lib):
    q, k = (9 * 256 + 3 * 64 + 64) * 2, (9 * 128 + 64 + 64) * 2
    cache = (4 * 512 + 3 * 128 + 64 + 64) * 2
    for form, spans in ((0, (q, k, 0, q, k, 0)), (1, (q, k, q, k, q, k)), (2, (q, k, k, q, cache, cache))):
        toks = (256, 128, 256 if form == 1 else 128, 128 if form == 1 else 256, 256 if form == 1 else 128, 128)
        st, h, _ = _plan(lib, "thd_qk_norm_rope_plan", _norm(form=form, bytes=spans, stride_tok=toks))
        assert st == 0
        lib.thd_attn_plan_destroy(h)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 1), (dict(page_size=0), 1), (dict(num_pages=-1), 1), (dict(max_pages=-1), 1), (dict(cap_rows=-1), 1),
    (dict(cap_free=-1), 1), (dict(table_stride=5), 1), (dict(flags=1), 1), (dict(batch=8193), 2),
    (dict(cap_rows=(1 << 21) + 1), 2), (dict(page_size=1 << 20, num_pages=1 << 11), 2),
    (dict(page_size=1 << 20, num_pages=1, max_pages=1 << 11, table_stride=1 << 11), 2),
])
def test_tables_descriptors_refused(lib, kw, code):
    assert _plan(lib, "thd_paged_tables_plan", _tables(**kw))[0] == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), 1), (dict(batch=-1), 1), (dict(h_q=3), 1), (dict(h_kv=0), 1), (dict(d=0), 1), (dict(page_size=0), 1),
    (dict(num_pages=-1), 1), (dict(table_stride=5), 1), (dict(stats_layout=2), 1), (dict(kernel=2), 1), (dict(kernel=4), 1),
    (dict(flags=1), 1), (dict(softmax_scale=float("inf")), 1), (dict(stride_page=(0, -1, 0, 0)), 1),
    (dict(d=136), 2), (dict(batch=8193), 2), (dict(page_size=1 << 20, num_pages=1 << 11), 2),
    (dict(dtype=2, kernel=3), 2), (dict(d=60, kernel=3), 2), (dict(kernel=3, stride_tok=(256, 132, 128, 256)), 2),
    (dict(bytes=(0, (19 * 512 + 3 * 128 + 64 + 64) * 2 - 2, 0, 0)), 4),
    (dict(bytes=((2 * 256 + 3 * 64 + 64) * 2 - 2, 0, 0, 0)), 4),
    # more work than the schedule can number
    (dict(batch=8192, h_q=4096, h_kv=4096, max_pages=1 << 20, table_stride=1 << 20, page_size=1024, num_pages=1), 2),
])
def test_decode_descriptors_refused(lib, kw, code):
    assert _plan(lib, "thd_paged_decode_plan", _decode(**kw))[0] == code


def test_decode_kernel_choice_and_sizes(lib):
    for kw, kernel in ((dict(), bd.KERNEL_MMA), (dict(dtype=1, d=8), bd.KERNEL_MMA), (dict(dtype=2), bd.KERNEL_SIMT),
                       (dict(d=60), bd.KERNEL_SIMT), (dict(kernel=1), bd.KERNEL_SIMT),
                       (dict(stride_head=(64, 68, 64, 64)), bd.KERNEL_SIMT)):
        st, h, ws = _plan(lib, "thd_paged_decode_plan", _decode(**kw))
        assert st == 0 and lib.thd_attn_plan_kernel(h) == kernel and ws % 256 == 0
        lib.thd_attn_plan_destroy(h)
    # the workspace goes by the GPU, not by the cache
    assert _plan(lib, "thd_paged_decode_plan", _decode(num_pages=1 << 20))[2] == \
        _plan(lib, "thd_paged_decode_plan", _decode())[2]


def test_calls_refused_before_launch(lib):
    """Wrong plan kind 1, missing pointers 1, missing or misaligned workspace 5, unaligned cache 3."""
    forms = [_plan(lib, "thd_qk_norm_rope_plan", _norm(form=f))[1] for f in range(3)]
    tables = _plan(lib, "thd_paged_tables_plan", _tables())[1]
    decode = _plan(lib, "thd_paged_decode_plan", _decode())[1]
    calls = {"thd_qk_norm_rope_fwd": (forms[0], 9), "thd_qk_norm_rope_bwd": (forms[1], 13),
             "thd_qk_norm_rope_paged": (forms[2], 12), "thd_paged_tables": (tables, 10), "thd_paged_decode": (decode, 9)}
    optional = {"thd_qk_norm_rope_fwd": {2, 3}, "thd_qk_norm_rope_bwd": {4, 5, 10, 11},
                "thd_qk_norm_rope_paged": {3, 4}, "thd_paged_tables": set(), "thd_paged_decode": {5, 7}}
    distinct = lambda n: [P * (i + 1) for i in range(n)]   # noqa: E731
    for name, (plan, n) in calls.items():
        fn = getattr(lib, name)
        for other in forms + [tables, decode, None]:
            if other is not plan:
                assert fn(other, *distinct(n), None) == 1, name
        for i in range(n):
            if i in optional[name]:
                continue
            args = distinct(n)
            args[i] = None
            assert fn(plan, *args, None) == (5 if i == n - 1 else 1), (name, i)
        args = distinct(n)
        args[-1] += 128
        assert fn(plan, *args, None) == 5, name
    args = distinct(9)
    args[1] += 8
    assert lib.thd_paged_decode(decode, *args, None) == 3
    # the page tables' inputs are not their outputs
    args = distinct(10)
    args[7] = args[0]
    assert lib.thd_paged_tables(tables, *args, None) == 1
    for where in (args[3], args[3] + 4):
        args = distinct(10)
        args[8] = where
        assert lib.thd_paged_tables(tables, *args, None) == 1
    # the attention entry points refuse these plans
    for plan in forms + [tables, decode]:
        assert lib.thd_attn_fwd(plan, *[P] * 15, None) == 1
        assert lib.thd_attn_bwd(plan, *[P] * 20, None) == 1
        assert lib.thd_indexer_topk(plan, *[P] * 13, None) == 1
        assert lib.thd_attn_fwd_static_ws(plan, *[P] * 14, None) == 1
        lib.thd_attn_plan_destroy(plan)


def test_plans_from_tensors_check_shapes():
    q, k = torch.zeros(6, 4, 64), torch.zeros(6, 2, 64)
    table = torch.zeros(10, 32)
    assert nr.qk_norm_rope_plan_for_tensors(q, k, q.clone(), k.clone(), table).workspace_bytes > 0
    for bad in (dict(k=k.half()), dict(q_out=q[:5]), dict(k_out=q), dict(q_out=q.transpose(1, 2)),
                dict(cos_sin=table.double()), dict(cos_sin=table[:, ::2])):
        args = dict(q=q, k=k, q_out=q.clone(), k_out=k.clone(), cos_sin=table)
        args.update(bad)
        with pytest.raises(ValueError):
            nr.qk_norm_rope_plan_for_tensors(**args)
    cache = torch.zeros(5, 4, 2, 64)
    with pytest.raises(ValueError):
        nr.qk_norm_rope_paged_plan_for_tensors(q, k, k, q, cache, cache[:, :3], table)
    bt = torch.zeros(6, 3, dtype=torch.int32)
    assert pg.paged_decode_plan_for_tensors(q, cache, cache, q, bt).kernel == bd.KERNEL_SIMT
    for bad in (dict(o=q[:5]), dict(v_cache=cache[:4]), dict(k_cache=cache.half()), dict(block_table=bt.long()),
                dict(block_table=bt[:5]), dict(q=q[..., :32], o=q[..., :32]), dict(block_table=bt[:1].expand(6, 3))):
        args = dict(q=q, k_cache=cache, v_cache=cache, o=q.clone(), block_table=bt)
        args.update(bad)
        with pytest.raises(ValueError):
            pg.paged_decode_plan_for_tensors(**args)


def test_one_call_functions_refuse_host_and_mistyped_tensors():
    q, k = torch.zeros(6, 4, 64), torch.zeros(6, 2, 64)
    w, table, pos = torch.ones(64), torch.zeros(10, 32), torch.zeros(6, dtype=torch.int32)
    cache, bt, lens = torch.zeros(5, 4, 2, 64), torch.zeros(6, 3, dtype=torch.int32), torch.zeros(6, dtype=torch.int32)
    cu = torch.zeros(7, dtype=torch.int32)
    calls = [
        lambda: rva.thd_qk_norm_rope_forward(q, k, w, w, table, pos),                  # host tensors
        lambda: rva.thd_qk_norm_rope_forward(q, k, w, w, table, pos.long()),
        lambda: rva.thd_qk_norm_rope_forward(q, k, w, w, table, pos[:5]),
        lambda: rva.thd_qk_norm_rope_forward(q, k, w[:32], w, table, pos),
        lambda: rva.thd_qk_norm_rope_forward(q, k, w.double(), w, table, pos),
        lambda: rva.thd_qk_norm_rope_append(q, k, k[:5], w, w, table, pos, pos, cache, cache),
        lambda: rva.thd_paged_attention(q, cache, cache, bt, lens),
        lambda: rva.thd_paged_attention(q, cache, cache, bt, lens.long()),
        lambda: rva.thd_paged_attention(q, cache, cache, bt, lens, window_left=lens[:2]),
        lambda: rva.thd_paged_attention(q, cache, cache, bt, lens, stats=torch.zeros(3)),
        lambda: rva.thd_paged_extend(lens, cu, lens, lens[:2].clone(), bt, page_size=4, num_pages=5),   # no rows
        lambda: rva.thd_paged_extend(lens, cu, lens, lens[:2].clone(), bt, page_size=4, num_pages=5, rows=4),
        lambda: rva.thd_paged_extend(lens, cu[:6], lens, lens[:2].clone(), bt, page_size=4, num_pages=5, rows=4),
        lambda: rva.thd_paged_extend(lens, cu, lens, lens[:2].clone(), bt.long(), page_size=4, num_pages=5, rows=4),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()
