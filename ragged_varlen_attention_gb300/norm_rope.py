"""Per-head RMS norm of Q and K with the position rotation (``thd_qk_norm_rope_*`` in
include/thd_attn.h): forward, backward, the serving form that fills the paged cache,
and the autograd function over the first two.

The functions that take a plan only marshal arguments, like ``thd_attn_fwd``; the
one-call functions check shapes, make the plan (cached) and allocate what is not given.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as _b

FORM_FWD, FORM_BWD, FORM_PAGED = 0, 1, 2
FLAG_ZERO_SKIPPED = 1 << 2
# the views (by index in the descriptor) that have Q's heads; the others have K's
_Q_VIEWS = {FORM_FWD: (0, 3), FORM_BWD: (0, 2, 4), FORM_PAGED: (0, 3)}


class ThdNormRopeDesc(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("form", ctypes.c_int),
        ("rows", ctypes.c_int32),
        ("h_q", ctypes.c_int32),
        ("h_kv", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("rot", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("max_pos", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("stride_tok", ctypes.c_int64 * 6),
        ("stride_head", ctypes.c_int64 * 6),
        ("stride_page", ctypes.c_int64 * 6),
        ("bytes", ctypes.c_int64 * 6),
        ("flags", ctypes.c_uint32),
    ]


def qk_norm_rope_plan(desc: ThdNormRopeDesc) -> _b.ThdAttnPlan:
    return _b.make_plan("thd_qk_norm_rope_plan", desc)


def _desc(form: int, views, cos_sin, eps: float, interleaved: bool, flags: int) -> ThdNormRopeDesc:
    """Descriptor from the six views of the form (None: unused); cache views are
    [pages, page_size, heads, d], the others [rows, heads, d]."""
    q, k = views[0], views[1]
    if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be a contiguous float32 [max_pos, rot] table")
    if q.dim() != 3 or k.dim() != 3 or q.dtype not in _b._DTYPE_CODE:
        raise ValueError("Q and K must be [rows, heads, d] of bfloat16, float16 or float32")
    desc = ThdNormRopeDesc()
    desc.dtype, desc.form = _b._DTYPE_CODE[q.dtype], form
    desc.rows, desc.h_q, desc.d = q.shape
    desc.h_kv = k.shape[1]
    desc.max_pos, desc.rot = cos_sin.shape
    desc.interleaved, desc.eps, desc.flags = int(interleaved), float(eps), int(flags)
    for i, t in enumerate(views):
        if t is None:
            continue
        cache = form == FORM_PAGED and i >= 4
        if t.dim() != (4 if cache else 3) or t.stride(-1) != 1:
            raise ValueError("Q, K, V and outputs must be [rows, heads, d] views, caches [pages, page_size, heads, d], "
                             "with a contiguous last dim")
        if t.dtype != q.dtype:
            raise ValueError("every view must share one storage type")
        heads = desc.h_q if i in _Q_VIEWS[form] else desc.h_kv
        if t.shape[-1] != desc.d or t.shape[-2] != heads or (not cache and t.shape[0] != desc.rows):
            raise ValueError(f"view {i} has shape {tuple(t.shape)}, which does not go with Q {tuple(q.shape)} and "
                             f"K {tuple(k.shape)}")
        if cache:
            if i == 4:
                desc.num_pages, desc.page_size = t.shape[0], t.shape[1]
            elif (desc.num_pages, desc.page_size) != tuple(t.shape[:2]):
                raise ValueError("the K and V caches must have the same pages")
            desc.stride_page[i] = t.stride(0)
        desc.stride_tok[i], desc.stride_head[i] = t.stride(-3), t.stride(-2)
        desc.bytes[i] = _b._view_bytes(t)
    return desc


def qk_norm_rope_plan_for_tensors(q, k, q_out, k_out, cos_sin, *, eps: float = 1e-6, interleaved: bool = False,
                                  flags: int = 0) -> _b.ThdAttnPlan:
    """Forward plan from [rows, heads, d] views (last dim contiguous) and the float32
    [max_pos, rot] table, whose width says how many elements of a head are rotated."""
    return qk_norm_rope_plan(_desc(FORM_FWD, (q, k, None, q_out, k_out, None), cos_sin, eps, interleaved, flags))


def qk_norm_rope_bwd_plan_for_tensors(q, k, dq_out, dk_out, dq, dk, cos_sin, *, eps: float = 1e-6,
                                      interleaved: bool = False, flags: int = 0) -> _b.ThdAttnPlan:
    """Backward plan from the forward's inputs, the upstream gradients and the gradients."""
    return qk_norm_rope_plan(_desc(FORM_BWD, (q, k, dq_out, dk_out, dq, dk), cos_sin, eps, interleaved, flags))


def qk_norm_rope_paged_plan_for_tensors(q, k, v, q_out, k_cache, v_cache, cos_sin, *, eps: float = 1e-6,
                                        interleaved: bool = False, flags: int = 0) -> _b.ThdAttnPlan:
    """Serving plan: caches are [pages, page_size, h_kv, d] views of any strides with a
    contiguous last dim (a [pages, h_kv, page_size, d] buffer is passed transposed)."""
    return qk_norm_rope_plan(_desc(FORM_PAGED, (q, k, v, q_out, k_cache, v_cache), cos_sin, eps, interleaved, flags))


def thd_qk_norm_rope_fwd(plan, q, k, w_q, w_k, cos_sin, positions, q_out, k_out, workspace, stream=None) -> None:
    """Enqueue the forward pass (see ``thd_qk_norm_rope_fwd`` in include/thd_attn.h)."""
    _b._enqueue("thd_qk_norm_rope_fwd", plan, q, (q, k, w_q, w_k, cos_sin, positions, q_out, k_out, workspace), stream)


def thd_qk_norm_rope_bwd(plan, q, k, dq_out, dk_out, w_q, w_k, cos_sin, positions, dq, dk, dw_q, dw_k, workspace,
                         stream=None) -> None:
    """Enqueue the backward pass (see ``thd_qk_norm_rope_bwd``); ``dw_q`` and ``dw_k`` are
    float32 [d] or None."""
    _b._enqueue("thd_qk_norm_rope_bwd", plan, q, (q, k, dq_out, dk_out, w_q, w_k, cos_sin, positions, dq, dk, dw_q, dw_k,
                                                  workspace), stream)


def thd_qk_norm_rope_paged(plan, q, k, v, w_q, w_k, cos_sin, positions, slot_map, q_out, k_cache, v_cache, workspace,
                           stream=None) -> None:
    """Enqueue the serving form (see ``thd_qk_norm_rope_paged``)."""
    _b._enqueue("thd_qk_norm_rope_paged", plan, q, (q, k, v, w_q, w_k, cos_sin, positions, slot_map, q_out, k_cache,
                                                    v_cache, workspace), stream)


# ----------------------------------------------------------------------- one-call functions
def _check(q, k, w_q, w_k, cos_sin, positions, slot_map=None):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("Q and K must be [rows, heads, d]")
    for w in (w_q, w_k):
        if w is not None and (w.shape != (q.shape[2],) or w.dtype != q.dtype or not w.is_contiguous()):
            raise ValueError("a weight must be a contiguous [d] tensor of Q's type, or None")
    for name, t in (("positions", positions), ("slot_map", slot_map)):
        if t is not None:
            _b._check_ints(name, t, (q.shape[0],))
    _b._check_devices(q, k, w_q, w_k, cos_sin, positions, slot_map)


def _key(kind, tensors, cos_sin, eps, interleaved, flags):
    return (kind, tuple((t.dtype, tuple(t.shape), t.stride(), _b._view_bytes(t)) for t in tensors), cos_sin.dtype,
            tuple(cos_sin.shape), cos_sin.stride(), eps, interleaved, flags)


def thd_qk_norm_rope_forward(q, k, w_q, w_k, cos_sin, positions, *, eps: float = 1e-6, interleaved: bool = False,
                             q_out=None, k_out=None, workspace=None, stream=None):
    """One-call forward. ``positions`` int32 [rows], negative for pad rows, which stay as
    they are in a given output and are zeros in one that is allocated here. Returns
    ``(q_out, k_out)``."""
    _check(q, k, w_q, w_k, cos_sin, positions)
    with _b._allocating_on(q, stream):
        flags = FLAG_ZERO_SKIPPED if q_out is None and k_out is None else 0
        fresh = torch.empty if flags else torch.zeros
        if q_out is None:
            q_out = fresh(q.shape, dtype=q.dtype, device=q.device)
        if k_out is None:
            k_out = fresh(k.shape, dtype=k.dtype, device=k.device)
        _b._check_devices(q, q_out, k_out)
        plan = _b._cached_plan(
            _key("norm_rope", (q, k, q_out, k_out), cos_sin, eps, interleaved, flags),
            lambda: qk_norm_rope_plan_for_tensors(q, k, q_out, k_out, cos_sin, eps=eps, interleaved=interleaved,
                                                  flags=flags))
        if workspace is None:
            workspace = _b.alloc_workspace(plan, q.device)
        thd_qk_norm_rope_fwd(plan, q, k, w_q, w_k, cos_sin, positions, q_out, k_out, workspace, stream)
    return q_out, k_out


def thd_qk_norm_rope_backward(q, k, dq_out, dk_out, w_q, w_k, cos_sin, positions, *, eps: float = 1e-6,
                              interleaved: bool = False, dq=None, dk=None, with_dw_q: bool = True,
                              with_dw_k: bool = True, workspace=None, stream=None):
    """One-call backward: the gradients of :func:`thd_qk_norm_rope_forward` for the
    upstream gradients ``dq_out`` and ``dk_out``. Returns ``(dq, dk, dw_q, dw_k)``, the
    last two float32 (None when not asked for)."""
    _check(q, k, w_q, w_k, cos_sin, positions)
    with _b._allocating_on(q, stream):
        flags = FLAG_ZERO_SKIPPED if dq is None and dk is None else 0
        fresh = torch.empty if flags else torch.zeros
        if dq is None:
            dq = fresh(q.shape, dtype=q.dtype, device=q.device)
        if dk is None:
            dk = fresh(k.shape, dtype=k.dtype, device=k.device)
        _b._check_devices(q, dq_out, dk_out, dq, dk)
        dw_q, dw_k = (torch.empty(q.shape[2], dtype=torch.float32, device=q.device) if wanted else None
                      for wanted in (with_dw_q, with_dw_k))
        plan = _b._cached_plan(
            _key("norm_rope_bwd", (q, k, dq_out, dk_out, dq, dk), cos_sin, eps, interleaved, flags),
            lambda: qk_norm_rope_bwd_plan_for_tensors(q, k, dq_out, dk_out, dq, dk, cos_sin, eps=eps,
                                                      interleaved=interleaved, flags=flags))
        if workspace is None:
            workspace = _b.alloc_workspace(plan, q.device)
        thd_qk_norm_rope_bwd(plan, q, k, dq_out, dk_out, w_q, w_k, cos_sin, positions, dq, dk, dw_q, dw_k, workspace,
                             stream)
    return dq, dk, dw_q, dw_k


def thd_qk_norm_rope_append(q, k, v, w_q, w_k, cos_sin, positions, slot_map, k_cache, v_cache, *, eps: float = 1e-6,
                            interleaved: bool = False, q_out=None, workspace=None, stream=None):
    """One-call serving form: K (normed, rotated) and V go to the rows of the paged cache
    that ``slot_map`` (int32 [rows], -1: nowhere) names. Returns Q, normed and rotated."""
    _check(q, k, w_q, w_k, cos_sin, positions, slot_map)
    if v.shape != k.shape:
        raise ValueError("V must have K's shape")
    with _b._allocating_on(q, stream):
        flags = FLAG_ZERO_SKIPPED if q_out is None else 0
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _b._check_devices(q, v, q_out, k_cache, v_cache)
        plan = _b._cached_plan(
            _key("norm_rope_paged", (q, k, v, q_out, k_cache, v_cache), cos_sin, eps, interleaved, flags),
            lambda: qk_norm_rope_paged_plan_for_tensors(q, k, v, q_out, k_cache, v_cache, cos_sin, eps=eps,
                                                        interleaved=interleaved, flags=flags))
        if workspace is None:
            workspace = _b.alloc_workspace(plan, q.device)
        thd_qk_norm_rope_paged(plan, q, k, v, w_q, w_k, cos_sin, positions, slot_map, q_out, k_cache, v_cache, workspace,
                               stream)
    return q_out


class ThdQkNormRope(torch.autograd.Function):
    """Per-head norm and rotation as an autograd function: ``thd_qk_norm_rope_fwd`` and
    ``thd_qk_norm_rope_bwd``. Use :func:`thd_qk_norm_rope`."""

    @staticmethod
    def forward(ctx, q, k, w_q, w_k, cos_sin, positions, eps, interleaved):
        q_out, k_out = thd_qk_norm_rope_forward(q, k, w_q, w_k, cos_sin, positions, eps=eps, interleaved=interleaved)
        ctx.save_for_backward(q, k, w_q, w_k, cos_sin, positions)
        ctx.eps, ctx.interleaved = eps, interleaved
        return q_out, k_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, w_q, w_k, cos_sin, positions = ctx.saved_tensors
        dq_out, dk_out = (t if t.stride(-1) == 1 else t.contiguous() for t in (dq_out, dk_out))
        need = ctx.needs_input_grad
        dq, dk, dw_q, dw_k = thd_qk_norm_rope_backward(
            q, k, dq_out, dk_out, w_q, w_k, cos_sin, positions, eps=ctx.eps, interleaved=ctx.interleaved,
            with_dw_q=need[2], with_dw_k=need[3])
        # the kernel sums in float32; the one rounding to a 16-bit weight's type is here
        return (dq, dk, dw_q.to(w_q.dtype) if need[2] else None, dw_k.to(w_k.dtype) if need[3] else None,
                None, None, None, None)


def thd_qk_norm_rope(q, k, w_q, w_k, cos_sin, positions, *, eps: float = 1e-6, interleaved: bool = False):
    """Differentiable per-head norm and rotation of Q [rows, h_q, d] and K [rows, h_kv, d]
    (see ``thd_qk_norm_rope_fwd`` in include/thd_attn.h), as :func:`thd_attention` reads
    them. Gradients flow to q, k, w_q and w_k; rows of negative position give zeros.

    Forward and backward may be captured into one CUDA graph. As for any backward pass that
    torch captures, drop the eager graphs over the same leaves first: torch accumulates into a
    leaf on the stream that its living graph was made on, which a capture does not allow."""
    return ThdQkNormRope.apply(q, k, w_q, w_k, cos_sin, positions, float(eps), bool(interleaved))
