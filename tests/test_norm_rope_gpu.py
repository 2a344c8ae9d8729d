"""The per-head norm with rotation on the GPU against the float64 oracle: forward,
backward, the serving form, the autograd function, and the calls that users make of
them (in place, on other streams, captured, with pad rows).

Tolerances, with u = 2^-24 (float32) and h = half a step of the storage type:
forward: the mean of squares is a sum of non-negative terms, at most 8 sequential
roundings, 5 in the shuffles and 2 more, so r is off by at most 10 u relative, and
rsqrt's own 2 u; y takes 2 more roundings and z 3, in all under 16 u (|y_a| + |y_b|);
the result is then rounded once: h |z| + 32 u (|y_a| + |y_b|).
backward: the same for g; dx = r (a - xh mean(a xh)) adds the mean's error, at most
32 u mean|a xh|, so 64 u r (|g_a| + |g_b|) |w| + 64 u r |xh| mean|a xh|, and h |dx|.
dw: terms g xh with at most 32 u each, added over fewer than 128 levels (4 heads a unit, the
units of a warp, the lanes, 8 warps, 38 blocks, 5 shuffles at these sizes): 160 u sum |g xh|.
float16 adds half its smallest step, 2^-25, for results below its normal range."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ragged_varlen_attention_gb300 as rva
from oracle import norm_rope_bwd, norm_rope_fwd
from ragged_varlen_attention_gb300 import binding as bd
from ragged_varlen_attention_gb300 import norm_rope as nr

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ragged_varlen_attention_gb300 import build
    build.build()
    bd.load_library()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def angles(max_pos, rot):
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def pair_sum(y, rot, interleaved):
    """|y_a| + |y_b| of each rotated element's pair, |y_e| elsewhere."""
    a = np.abs(y)
    out = a.copy()
    half = rot // 2
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out[..., ia] = out[..., ib] = a[..., ia] + a[..., ib]
    return out


def fwd_bound(x, w, rot, interleaved, eps, dtype, z):
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return HALF[dtype] * np.abs(z) + TINY[dtype] + 32 * U * pair_sum(y, rot, interleaved)


def make(seed, rows, h_q, h_kv, d, rot, dtype, pad=True, max_pos=500):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    qkv = rand(rows, h_q + 2 * h_kv, d)
    q, k, v = qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:]
    w_q, w_k = (1 + 0.25 * torch.randn(d, generator=g, device="cuda")).to(dtype), rand(d)
    pos = torch.randint(0, max_pos, (rows,), generator=g, device="cuda").int()
    if pad and rows > 2:
        pos[rows // 2] = -1
        pos[-1] = -7
    return q, k, v, w_q, w_k, angles(max_pos, rot), pos


SHAPES = [
    # rows, h_q, h_kv, d, rot, interleaved, dtype
    (1, 1, 1, 8, 8, False, torch.bfloat16),
    (37, 32, 8, 128, 128, False, torch.bfloat16),
    (37, 5, 1, 128, 64, True, torch.float16),
    (29, 16, 16, 64, 32, True, torch.float16),
    (29, 16, 2, 64, 64, False, torch.bfloat16),
    (23, 20, 4, 96, 96, False, torch.float32),
    (23, 7, 1, 80, 40, False, torch.float32),
    (11, 3, 3, 256, 128, False, torch.bfloat16),
    (11, 3, 1, 200, 200, True, torch.float32),
    (19, 9, 3, 24, 0, False, torch.float16),       # no rotation at all
    (19, 4, 2, 33, 10, False, torch.float32),      # the kernel for any size
    (19, 4, 2, 57, 56, True, torch.bfloat16),
    (19, 4, 2, 128, 12, False, torch.bfloat16),    # rot not a multiple of 8
    (7, 2, 2, 1, 0, False, torch.float32),
    (7, 2, 1, 2, 2, True, torch.float16),
    (3000, 4, 2, 64, 64, False, torch.bfloat16),   # units wrap around the grid
]


@pytest.mark.parametrize("rows,h_q,h_kv,d,rot,interleaved,dtype", SHAPES)
def test_forward(rows, h_q, h_kv, d, rot, interleaved, dtype):
    eps = 1e-6
    q, k, _, w_q, w_k, table, pos = make(rows + d, rows, h_q, h_kv, d, rot, dtype)
    q_out, k_out = (torch.full(t.shape, 7.0, dtype=dtype, device="cuda") for t in (q, k))
    rva.thd_qk_norm_rope_forward(q, k, w_q, w_k, table, pos, eps=eps, interleaved=interleaved, q_out=q_out, k_out=k_out)
    live = f64(pos) >= 0
    for x, w, out in ((q, w_q, q_out), (k, w_k, k_out)):
        ref = norm_rope_fwd(f64(x), f64(w), f64(table), pos.cpu().numpy(), eps, interleaved, np.full(x.shape, 7.0))
        got = f64(out)
        assert (got[~live] == 7.0).all()
        bound = fwd_bound(f64(x), f64(w), rot, interleaved, eps, dtype, ref)
        assert (np.abs(got - ref) <= bound)[live].all(), np.max((np.abs(got - ref) - bound)[live])


@pytest.mark.parametrize("rows,h_q,h_kv,d,rot,interleaved,dtype", SHAPES)
def test_backward(rows, h_q, h_kv, d, rot, interleaved, dtype):
    eps = 1e-5
    q, k, _, w_q, w_k, table, pos = make(2 * rows + d, rows, h_q, h_kv, d, rot, dtype)
    g = torch.Generator(device="cuda").manual_seed(9)
    dq_out, dk_out = (torch.randn(t.shape, generator=g, device="cuda").to(dtype) for t in (q, k))
    dq, dk = (torch.full(t.shape, 7.0, dtype=dtype, device="cuda") for t in (q, k))
    got = rva.thd_qk_norm_rope_backward(q, k, dq_out, dk_out, w_q, w_k, table, pos, eps=eps, interleaved=interleaved,
                                        dq=dq, dk=dk)
    live = f64(pos) >= 0
    p = pos.cpu().numpy()
    for x, w, dz, dx, dw in ((q, w_q, dq_out, got[0], got[2]), (k, w_k, dk_out, got[1], got[3])):
        x, w, dz = f64(x), f64(w), f64(dz)
        ref, ref_w = norm_rope_bwd(x, dz, w, f64(table), p, eps, interleaved, np.full(x.shape, 7.0))
        assert (f64(dx)[~live] == 7.0).all()
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        size = pair_sum(dz, rot, interleaved)   # bounds |g| of the pair up to the rotation
        xh = np.abs(x) * r
        bound = HALF[dtype] * np.abs(ref) + TINY[dtype] + 64 * U * r * (
            size * np.abs(w) + xh * (size * np.abs(w) * xh).mean(-1, keepdims=True))
        err = np.abs(f64(dx) - ref)
        assert (err <= bound)[live].all(), np.max((err - bound)[live])
        assert (np.abs(f64(dw) - ref_w) <= 160 * U * (size * xh)[live].sum((0, 1))).all()


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("h_q,h_kv,d,rot,dtype", [(8, 2, 128, 128, torch.bfloat16), (6, 3, 64, 32, torch.float16),
                                                  (4, 4, 96, 96, torch.float32), (5, 1, 33, 10, torch.float32)])
def test_paged_form(h_q, h_kv, d, rot, dtype, page, heads_first):
    rows, eps = 41, 1e-6
    q, k, v, w_q, w_k, table, pos = make(page + d, rows, h_q, h_kv, d, rot, dtype)
    pages = -(-rows // page) + 3
    shape = (pages, h_kv, page, d) if heads_first else (pages, page, h_kv, d)
    caches = [torch.full(shape, 3.0, dtype=dtype, device="cuda") for _ in range(2)]
    views = [c.transpose(1, 2) if heads_first else c for c in caches]
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(5))[:rows].int().cuda()
    slots[3] = -1
    q_out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    rva.thd_qk_norm_rope_append(q, k, v, w_q, w_k, table, pos, slots, views[0], views[1], eps=eps, q_out=q_out)
    p, s = pos.cpu().numpy(), slots.cpu().numpy()
    ref_q = norm_rope_fwd(f64(q), f64(w_q), f64(table), p, eps, False, np.full(q.shape, 7.0))
    ref_k = norm_rope_fwd(f64(k), f64(w_k), f64(table), p, eps, False, np.zeros(k.shape))
    assert (np.abs(f64(q_out) - ref_q) <= fwd_bound(f64(q), f64(w_q), rot, False, eps, dtype, ref_q)).all()
    bound_k = fwd_bound(f64(k), f64(w_k), rot, False, eps, dtype, ref_k)
    got_k, got_v = (f64(c).reshape(pages * page, h_kv, d) for c in views)
    written = np.zeros(pages * page, dtype=bool)
    for t in range(rows):
        if p[t] >= 0 and s[t] >= 0:
            written[s[t]] = True
            assert (np.abs(got_k[s[t]] - ref_k[t]) <= bound_k[t]).all()
            assert np.array_equal(got_v[s[t]], f64(v)[t])
    assert written.sum() == rows - 3
    assert (got_k[~written] == 3.0).all() and (got_v[~written] == 3.0).all()


def test_status_of_bad_positions_and_slots():
    q, k, v, w_q, w_k, table, pos = make(3, 9, 4, 2, 64, 64, torch.bfloat16, pad=False, max_pos=50)
    pos[2] = 50
    q_out, k_out = (torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda") for t in (q, k))
    plan = rva.qk_norm_rope_plan_for_tensors(q, k, q_out, k_out, table)
    ws = rva.alloc_workspace(plan, "cuda")
    rva.thd_qk_norm_rope_fwd(plan, q, k, w_q, w_k, table, pos, q_out, k_out, ws)
    assert rva.thd_attn_read_status(plan, ws) == bd.DEV_BAD_POSITION
    assert (q_out[2] == 7).all() and (k_out[2] == 7).all() and (q_out[3] != 7).any()
    pos[2] = 49
    rva.thd_qk_norm_rope_fwd(plan, q, k, w_q, w_k, table, pos, q_out, k_out, ws)
    assert rva.thd_attn_read_status(plan, ws) == 0 and (q_out[2] != 7).any()
    cache = torch.full((2, 3, 4, 2, 64), 3.0, dtype=q.dtype, device="cuda")
    plan = rva.qk_norm_rope_paged_plan_for_tensors(q, k, v, q_out, cache[0], cache[1], table)
    ws = rva.alloc_workspace(plan, "cuda")
    slots = torch.tensor([0, 1, 2, 12, 11, -1, -2 ** 31, 2 ** 31 - 1, 5], dtype=torch.int32, device="cuda")
    rva.thd_qk_norm_rope_paged(plan, q, k, v, w_q, w_k, table, pos, slots, q_out, cache[0], cache[1], ws)
    assert rva.thd_attn_read_status(plan, ws) == bd.DEV_BAD_PAGE
    got = (cache.view(2, 12, -1) != 3).any(-1).any(0).nonzero().flatten().tolist()
    assert got == [0, 1, 2, 5, 11]


@pytest.mark.parametrize("d,rot", [(128, 128), (48, 20)])
def test_weights_may_be_absent_and_zero_rows_are_zero(d, rot):
    """No weight stands for ones; a head of zeros gives zeros for any eps > 0; rows that are
    skipped are zeros in outputs that the call makes, the gradients among them."""
    q, k, _, _, _, table, pos = make(8, 21, 3, 3, d, rot, torch.float32)
    q, k = q.clone(), k.clone()
    q[4] = 0
    ones = torch.ones(d, device="cuda")
    a = rva.thd_qk_norm_rope_forward(q, k, None, None, table, pos)
    b = rva.thd_qk_norm_rope_forward(q, k, ones, ones, table, pos)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    skipped = (pos < 0).nonzero().flatten()
    assert (a[0][4] == 0).all() and (a[0][skipped] == 0).all() and (a[1][skipped] == 0).all()
    dz = torch.randn(q.shape, device="cuda")
    dq, dk, dw_q, dw_k = rva.thd_qk_norm_rope_backward(q, k, dz, dz, None, None, table, pos, with_dw_k=False)
    assert dw_k is None and torch.isfinite(dq).all() and torch.isfinite(dw_q).all()
    assert (dq[skipped] == 0).all() and (dk[skipped] == 0).all()


def test_a_nan_row_stays_in_its_head_and_pad_rows_may_hold_anything():
    q, k, _, w_q, w_k, table, pos = make(13, 17, 4, 2, 64, 64, torch.bfloat16)
    q, k = q.clone(), k.clone()
    clean = rva.thd_qk_norm_rope_forward(q, k, w_q, w_k, table, pos)
    dz = [torch.randn(t.shape, device="cuda").to(t.dtype) for t in (q, k)]
    clean_g = rva.thd_qk_norm_rope_backward(q, k, dz[0], dz[1], w_q, w_k, table, pos)
    q[pos < 0] = float("nan")
    k[pos < 0] = float("inf")
    dz[0][pos < 0] = float("nan")
    got = rva.thd_qk_norm_rope_forward(q, k, w_q, w_k, table, pos)
    assert all(torch.equal(a, b) for a, b in zip(got, clean))
    assert all(torch.equal(a, b) for a, b in zip(rva.thd_qk_norm_rope_backward(q, k, dz[0], dz[1], w_q, w_k, table, pos),
                                                 clean_g))
    q[3, 1, 5] = float("nan")
    got = rva.thd_qk_norm_rope_forward(q, k, w_q, w_k, table, pos)
    assert got[0][3, 1].isnan().all()
    got[0][3, 1] = clean[0][3, 1]
    assert torch.equal(got[0], clean[0])


def test_in_place():
    q, k, _, w_q, w_k, table, pos = make(17, 50, 8, 2, 128, 64, torch.bfloat16)
    q, k = q.clone(), k.clone()
    out = [torch.empty_like(t).copy_(t) for t in (q, k)]
    rva.thd_qk_norm_rope_forward(q, k, w_q, w_k, table, pos, q_out=out[0], k_out=out[1])
    rva.thd_qk_norm_rope_forward(q, k, w_q, w_k, table, pos, q_out=q, k_out=k)
    assert torch.equal(q, out[0]) and torch.equal(k, out[1])


@pytest.mark.parametrize("d,rot", [(128, 128), (57, 12)])
def test_backward_in_place(d, rot):
    q, k, _, w_q, w_k, table, pos = make(18, 333, 8, 2, d, rot, torch.float32)
    dz = [torch.randn(t.shape, device="cuda") for t in (q, k)]
    keep = [t.clone() for t in dz]
    ref = rva.thd_qk_norm_rope_backward(q, k, *keep, w_q, w_k, table, pos, dq=dz[0].clone(), dk=dz[1].clone())
    got = rva.thd_qk_norm_rope_backward(q, k, *dz, w_q, w_k, table, pos, dq=dz[0], dk=dz[1])
    assert got[0] is dz[0] and all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("h_q,h_kv,d", [(8, 8, 128), (16, 4, 128), (6, 3, 64), (16, 16, 64), (5, 5, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_units_that_span_tokens_and_units_of_one(h_q, h_kv, d, dtype):
    """More rows than the grid takes at once, for each division of heads into units: every row is
    the row that a call on it alone gives."""
    rows = 5003
    q, k, _, w_q, w_k, table, pos = make(rows, rows, h_q, h_kv, d, d, dtype)
    out = rva.thd_qk_norm_rope_forward(q, k, w_q, w_k, table, pos)
    dz = [torch.randn(t.shape, device="cuda").to(dtype) for t in (q, k)]
    grads = rva.thd_qk_norm_rope_backward(q, k, dz[0], dz[1], w_q, w_k, table, pos)
    some = torch.tensor([0, 1, 777, rows // 2, 2501, rows - 2, rows - 1], device="cuda")
    a = rva.thd_qk_norm_rope_forward(q[some], k[some], w_q, w_k, table, pos[some])
    b = rva.thd_qk_norm_rope_backward(q[some], k[some], dz[0][some], dz[1][some], w_q, w_k, table, pos[some])
    for whole, part in zip(out + grads[:2], a + b[:2]):
        assert torch.equal(whole[some], part)
    # dw over everything: sums of 5003 x heads terms of at most u(32) each, over fewer than 256 levels
    for x, z, w, dw in ((q, dz[0], w_q, grads[2]), (k, dz[1], w_k, grads[3])):
        live = (pos >= 0).cpu().numpy()
        xs, zs = f64(x), f64(z)
        _, ref = norm_rope_bwd(xs, zs, f64(w), f64(table), pos.cpu().numpy(), 1e-6, False, np.zeros(x.shape))
        xh = np.abs(xs) / np.sqrt((xs * xs).mean(-1, keepdims=True) + 1e-6)
        bound = 288 * U * (pair_sum(zs, d, False) * xh)[live].sum((0, 1))
        assert (np.abs(f64(dw) - ref) <= bound).all()


def test_vector_and_any_size_kernels_agree():
    """The same values through views that allow wide accesses and through views that do not."""
    q, k, _, w_q, w_k, table, pos = make(19, 40, 6, 2, 64, 32, torch.bfloat16)
    odd = [torch.empty(t.shape[0], t.shape[1], 65, dtype=t.dtype, device="cuda")[..., :64].copy_(t) for t in (q, k)]
    a, b = (rva.thd_qk_norm_rope_forward(*x, w_q, w_k, table, pos) for x in ((q, k), odd))
    for s, t in zip(a, b):   # both are within the tolerance of the exact result
        assert (s.float() - t.float()).abs().max() <= 2 * 2.0 ** -8 * s.float().abs().max()


def test_autograd_chain_with_attention():
    """q, k, v -> norm and rotation -> packed attention -> gradients of projections and weights,
    against the composed oracles; broadcast upstream gradients and shared weights included."""
    from oracle import thd_attention_bwd, thd_attention_fwd
    h_q, h_kv, d, eps = 4, 2, 64, 1e-6
    lens = [30, 41]
    cu = np.array([0, 30, 71], dtype=np.int32)
    q, k, v, w, _, table, _ = make(23, 71, h_q, h_kv, d, d, torch.float32, pad=False)
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    leaves = [t.detach().clone().requires_grad_(True) for t in (q, k, v, w)]
    qz, kz = rva.thd_qk_norm_rope(leaves[0], leaves[1], leaves[3], leaves[3], table, pos, eps=eps)
    cud = torch.from_numpy(cu).cuda()
    mask = torch.tensor([1, 2], dtype=torch.int8, device="cuda")
    o = rva.thd_attention(qz, kz, leaves[2], cud, cud, mask_type=mask)
    up = torch.randn(o.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    (o * up).sum().backward()
    p = pos.cpu().numpy()
    zero = lambda t: np.zeros(tuple(t.shape))  # noqa: E731
    rq, rk = (norm_rope_fwd(f64(t), f64(w), f64(table), p, eps, False, zero(t)) for t in (q, k))
    off = cu[:-1]
    ro, _, _ = thd_attention_fwd(rq, rk, f64(v), cu, cu, off, off, off, off, off, np.array([1, 2]), None, zero(q),
                                 np.zeros(71 * h_q), h_q, 1)
    dq, dk, dv, *_ = thd_attention_bwd(rq, rk, f64(v), f64(up), cu, cu, off, off, off, off, np.array([1, 2]), None,
                                       zero(q), zero(k), zero(v))
    gq, gw = norm_rope_bwd(f64(q), dq, f64(w), f64(table), p, eps, False, zero(q))
    gk, gw2 = norm_rope_bwd(f64(k), dk, f64(w), f64(table), p, eps, False, zero(k))
    assert np.abs(f64(o) - ro).max() <= 1e-4    # the float32 attention's own bound
    for got, ref in ((leaves[0].grad, gq), (leaves[1].grad, gk), (leaves[2].grad, dv), (leaves[3].grad, gw + gw2)):
        assert np.abs(f64(got) - ref).max() <= 1e-4 * max(1.0, np.abs(ref).max())


def test_autograd_takes_broadcast_gradients_and_unused_outputs():
    q, k, _, w_q, w_k, table, pos = make(29, 20, 4, 2, 64, 64, torch.float32)
    q, k, w_q = (t.detach().clone().requires_grad_(True) for t in (q, k, w_q))
    qz, kz = rva.thd_qk_norm_rope(q, k, w_q, w_k, table, pos)
    qz.sum().backward()      # a gradient of strides 0; none for K's output
    ones = torch.ones(q.shape, device="cuda")
    ref = rva.thd_qk_norm_rope_backward(q.detach(), k.detach(), ones, torch.zeros(k.shape, device="cuda"), w_q.detach(),
                                        w_k, table, pos)
    assert torch.equal(q.grad, ref[0]) and (k.grad == 0).all() and torch.equal(w_q.grad, ref[2])


def test_gradients_match_differences():
    """Directional differences of the kernels' own forward, float32."""
    q, k, _, w_q, w_k, table, pos = make(31, 6, 2, 1, 32, 16, torch.float32)
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda t: torch.randn(t.shape, generator=g, device="cuda")  # noqa: E731
    uq, uk = rand(q), rand(k)
    loss = lambda a, b, c, e: sum(float((z.double() * u.double()).sum()) for z, u in  # noqa: E731
                                  zip(rva.thd_qk_norm_rope_forward(a, b, c, e, table, pos), (uq, uk)))
    grads = rva.thd_qk_norm_rope_backward(q, k, uq, uk, w_q, w_k, table, pos)
    args = [q, k, w_q, w_k]
    for i in range(4):
        direction = rand(args[i])
        step = 2.0 ** -8
        up, down = ([t + s * direction if j == i else t for j, t in enumerate(args)] for s in (step, -step))
        diff = (loss(*up) - loss(*down)) / (2 * step)
        want = float((grads[i].double() * direction.double()).sum())
        # the difference's own error: a third derivative of order one in step^2, and float32 losses
        # of fewer than 600 terms over 2 step; both under 2^-8 of the gradient's size
        assert abs(diff - want) <= 2.0 ** -8 * float((grads[i].double().abs() * direction.double().abs()).sum()), i


def test_equal_inputs_give_equal_bits_and_graph_replays_see_new_inputs():
    q, k, _, w_q, w_k, table, pos = make(37, 700, 8, 2, 128, 128, torch.bfloat16)
    dz = [torch.randn(t.shape, device="cuda").to(t.dtype) for t in (q, k)]
    a = rva.thd_qk_norm_rope_backward(q, k, dz[0], dz[1], w_q, w_k, table, pos)
    b = rva.thd_qk_norm_rope_backward(q, k, dz[0], dz[1], w_q, w_k, table, pos)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    xq, xk = q.clone(), k.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rva.thd_qk_norm_rope_forward(xq, xk, w_q, w_k, table, pos)
        grads = rva.thd_qk_norm_rope_backward(xq, xk, dz[0], dz[1], w_q, w_k, table, pos)
    xq.mul_(-1.5)
    graph.replay()
    ref = rva.thd_qk_norm_rope_forward(xq, xk, w_q, w_k, table, pos)
    ref_g = rva.thd_qk_norm_rope_backward(xq, xk, dz[0], dz[1], w_q, w_k, table, pos)
    assert all(torch.equal(s, t) for s, t in zip(out + grads, ref + ref_g))


def test_a_captured_training_step_replays():
    """Forward and backward through autograd and packed attention in one CUDA graph, after a
    warm-up on a side stream whose eager graph is gone; against the same step made eagerly."""
    h_q, h_kv, d = 4, 2, 64
    x, y, v, w, _, table, _ = make(47, 90, h_q, h_kv, d, d, torch.bfloat16, pad=False)
    pos = torch.arange(90, device="cuda").int() % 45
    cu, mask = torch.tensor([0, 45, 90], dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int8, device="cuda")
    leaves = [t.detach().clone().requires_grad_(True) for t in (x, y, v, w)]

    def step():
        qz, kz = rva.thd_qk_norm_rope(leaves[0], leaves[1], leaves[3], leaves[3], table, pos)
        o = rva.thd_attention(qz, kz, leaves[2], cu, cu, mask_type=mask)
        return torch.autograd.grad(o.float().square().sum(), leaves)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.no_grad():
        leaves[0].mul_(-0.5)
        leaves[3].add_(0.25)
    graph.replay()
    ref = step()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_on_a_given_stream():
    q, k, _, w_q, w_k, table, pos = make(41, 300, 8, 2, 128, 128, torch.bfloat16)
    ref = rva.thd_qk_norm_rope_forward(q, k, w_q, w_k, table, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = rva.thd_qk_norm_rope_forward(q, k, w_q, w_k, table, pos, stream=s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_on_the_current_stream():
    q, k, _, w_q, w_k, table, pos = make(42, 300, 8, 2, 128, 128, torch.bfloat16)
    ref = rva.thd_qk_norm_rope_forward(q, k, w_q, w_k, table, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        late = q.clone().mul_(1)     # made on the side stream: the call has to come after it
        got = rva.thd_qk_norm_rope_forward(late, k, w_q, w_k, table, pos)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_no_rows():
    q, k, v, w_q, w_k, table, pos = make(43, 1, 4, 2, 64, 64, torch.bfloat16)
    q, k, v, pos = q[:0], k[:0], v[:0], pos[:0]
    assert rva.thd_qk_norm_rope_forward(q, k, w_q, w_k, table, pos)[0].shape == (0, 4, 64)
    got = rva.thd_qk_norm_rope_backward(q, k, q, k, w_q, w_k, table, pos)
    assert (got[2] == 0).all() and (got[3] == 0).all()
    plan = rva.qk_norm_rope_plan_for_tensors(q, k, q, k, table)
    ws = torch.full((plan.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")
    rva.thd_qk_norm_rope_fwd(plan, q, k, w_q, w_k, table, pos, q, k, ws)
    assert rva.thd_attn_read_status(plan, ws) == 0


def test_rows_past_32_bits_of_elements():
    """Token strides that put the last rows past 2^31 elements of the view."""
    h, d = 2, 64
    rows, stride = 9, (1 << 28) + 64
    big = torch.empty((rows - 1) * stride + h * d, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((rows, h, d), (stride, d, 1))
    g = torch.Generator(device="cuda").manual_seed(1)
    q.copy_(torch.randn((rows, h, d), generator=g, device="cuda"))
    k = torch.randn((rows, h, d), generator=g, device="cuda").to(torch.bfloat16)
    table, pos = angles(16, d), torch.arange(rows, device="cuda").int()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    a = rva.thd_qk_norm_rope_forward(q, k, w, w, table, pos)
    b = rva.thd_qk_norm_rope_forward(q.contiguous(), k, w, w, table, pos)
    assert torch.equal(a[0], b[0])
    assert nr.FLAG_ZERO_SKIPPED == 4
