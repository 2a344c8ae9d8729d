"""The oracles of the norm with rotation and of the paged cache, pinned to facts outside
themselves: closed forms, differences, invariants, and the packed attention oracle."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import norm_rope_bwd, norm_rope_fwd, paged_attention, paged_tables, thd_attention_fwd


def _table(max_pos, rot):
    a = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    return np.concatenate([np.cos(a), np.sin(a)], 1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_sees_relative_positions(interleaved):
    rng = np.random.default_rng(3)
    d, table = 16, _table(40, 16)
    x = np.repeat(rng.standard_normal((1, 2, d)), 40, axis=0)
    z = norm_rope_fwd(x, None, table, np.arange(40), 0.0, interleaved, np.zeros_like(x))
    # eps = 0: every head has mean square one, and a rotation keeps it
    assert np.allclose((z * z).mean(-1), 1.0, atol=1e-12)
    # <R(p) a, R(p') b> depends on p - p' alone
    assert np.allclose(z[3, 0] @ z[10, 1], z[20, 0] @ z[27, 1], atol=1e-12)
    # position 0 turns nothing
    assert np.allclose(z[0], x[0] / np.sqrt((x[0] ** 2).mean(-1, keepdims=True)), atol=1e-14)


def test_layouts_are_permutations_of_each_other():
    rng = np.random.default_rng(4)
    table = _table(9, 8)
    x = rng.standard_normal((9, 1, 12))
    order = np.r_[np.stack([np.arange(4), np.arange(4) + 4], 1).ravel(), 8:12]   # halves -> adjacent
    a = norm_rope_fwd(x, None, table, np.arange(9), 1e-6, False, np.zeros_like(x))
    b = norm_rope_fwd(x[..., order], None, table, np.arange(9), 1e-6, True, np.zeros_like(x))
    assert np.allclose(a[..., order], b, atol=1e-14)


@pytest.mark.parametrize("interleaved,rot", [(False, 8), (True, 4), (False, 0)])
def test_backward_matches_differences(interleaved, rot):
    rng = np.random.default_rng(5)
    rows, heads, d, eps = 4, 2, 8, 1e-3
    table, pos = _table(30, rot), np.array([3, -1, 29, 7])
    x, w, dz = rng.standard_normal((rows, heads, d)), 1 + 0.3 * rng.standard_normal(d), rng.standard_normal((rows, heads, d))
    f = lambda x_, w_: float((norm_rope_fwd(x_, w_, table, pos, eps, interleaved, np.zeros_like(x)) * dz).sum())  # noqa: E731
    dx, dw = norm_rope_bwd(x, dz, w, table, pos, eps, interleaved, np.zeros_like(x))
    h = 1e-5
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-8
    for i in range(d):
        e = np.zeros(d)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-8
    assert (dx[1] == 0).all()   # the pad row


def test_paged_attention_is_the_last_row_of_packed_attention():
    rng = np.random.default_rng(6)
    lens, h_q, h_kv, d, page = [1, 7, 20, 0], 4, 2, 8, 3
    cu = np.concatenate([[0], np.cumsum(lens)])
    k, v = rng.standard_normal((2, cu[-1], h_kv, d))
    q = rng.standard_normal((4, h_q, d))
    k_cache, v_cache = (np.full((12, page, h_kv, d), np.nan) for _ in range(2))
    order, table, at = rng.permutation(12), np.full((4, 7), -1), 0
    for b, n in enumerate(lens):
        for j in range(n):
            if j % page == 0:
                table[b, j // page] = order[at]
                at += 1
            k_cache[table[b, j // page], j % page] = k[cu[b] + j]
            v_cache[table[b, j // page], j % page] = v[cu[b] + j]
    for window in (None, [0, 2, 100, 5]):
        o, lse, status = paged_attention(q, k_cache, v_cache, table, lens, 0.3, window)
        assert status == 0
        cu_q = np.arange(5)
        ref_o, ref_s, _ = thd_attention_fwd(q, k, v, cu_q, cu, cu_q[:-1], cu[:-1], cu[:-1], cu_q[:-1], cu_q[:-1],
                                            np.full(4, 2), None, np.zeros_like(q), np.zeros(16), 4, 1,
                                            softmax_scale=0.3, window_left=None if window is None else np.array(window))
        assert np.allclose(o, ref_o, atol=1e-13)
        assert np.allclose(lse.ravel()[:12], ref_s[:12], atol=1e-13) and np.isneginf(lse[3]).all()


def test_paged_tables_by_hand():
    # pages of 4; request 0 has 3 tokens in page 9 and gets 6; 1 has none and gets none; 2 has 4 in page 5 and gets 1
    table = np.array([[9, -1, -1], [-1, -1, -1], [5, -1, -1]])
    got = paged_tables([3, 0, 4], [0, 6, 6, 7], [7, 2, 8, 1], [0, 4], table, 4, 10, 8)
    assert got[0].tolist() == [[9, 7, 2], [-1, -1, -1], [5, 8, -1]]
    assert got[1].tolist() == [39, 28, 29, 30, 31, 8, 32, -1]
    assert got[2].tolist() == [3, 4, 5, 6, 7, 8, 4, -1]
    assert got[3].tolist() == [9, 0, 5] and got[4] == 3 and got[5] == 0
    # with two free pages the last request stays as long as it was
    got = paged_tables([3, 0, 4], [0, 6, 6, 7], [7, 2], [0, 2], table, 4, 10, 8)
    assert got[0][2].tolist() == [5, -1, -1] and got[1][6] == -1 and got[3].tolist() == [9, 0, 4]
    assert got[4] == 2 and got[5] == 128
