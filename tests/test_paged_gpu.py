"""Page tables and one-token attention over pages on the GPU against the oracles, and the
serving step that they form with the norm-with-rotation's paged form.

Page tables are whole numbers and have to be equal. Tolerance of the attention, with
u = 2^-24, h = half a step of the storage type, M = max_j scale sum_e |q_e k_je|:
a score is a float32 sum of exact products (16-bit inputs; float32 ones round once more)
that the tensor core adds in steps of 16 with at most a few truncated bits each, and one
product with the scale: off by at most 64 u M. exp2 and the running rescaling add a few u
each time a maximum moves, and a sum of n terms at most (n / 64 + 64) u: with
e = 64 u M + (n / 64 + 96) u the weights p are off by e relative, and so is Stats, plus its
own rounding, 4 u |Stats|. The matrix kernel takes p as two 16-bit parts (what is left is h^2,
and half of float16's smallest step, 2^-25, for each key). So O is off by at most
h |O| + (h^2 + 2 e) sum_j p_j |v_j| + n 2^-25 max|v| (float16)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ragged_varlen_attention_gb300 as rva
from oracle import norm_rope_fwd, paged_attention, paged_tables
from ragged_varlen_attention_gb300 import binding as bd

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ragged_varlen_attention_gb300 import build
    build.build()
    bd.load_library()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------- page tables
def run_tables(lens, new, page, pages, cols, free, span=None, rows=None, table=None, cu=None, stride=None):
    """One call and the oracle on the same inputs; every output and the status compared."""
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int64) if cu is None else np.array(cu)
    rows = int(cu[-1]) if rows is None else rows
    span = [0, len(free)] if span is None else span
    if table is None:
        table = np.arange(len(lens) * cols).reshape(len(lens), cols) % max(pages, 1)
    backing = torch.full((max(len(lens), 1), stride or cols), -5, dtype=torch.int32, device="cuda")
    dev = backing[:len(lens), :cols]
    dev.copy_(ints(table.tolist()).view(len(lens), cols))
    plan = rva.paged_tables_plan(len(lens), page, pages, cols, stride or cols, rows, len(free))
    ws = torch.full((plan.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")
    out = [torch.full((n + 8,), -9, dtype=torch.int32, device="cuda") for n in (rows, rows, len(lens), 1)]
    inputs = [ints(list(v)) for v in (lens, cu, free, span)]
    for _ in range(2):   # a repeated call gives the same
        rva.thd_paged_tables(plan, inputs[0], inputs[1], inputs[2], inputs[3], dev, *out, ws)
    status = rva.thd_attn_read_status(plan, ws)
    ref = paged_tables(lens, cu, free, span, table, page, pages, rows)
    assert status == ref[5]
    assert np.array_equal(dev.cpu().numpy().reshape(len(lens), cols), ref[0])
    for got, want in zip(out, ref[1:5]):
        want = np.atleast_1d(want)
        assert np.array_equal(got.cpu().numpy()[:len(want)], want)
        assert (got[len(want):] == -9).all()
    assert (backing[:, cols:] == -5).all()
    return ref


@pytest.mark.parametrize("batch,mean,new,page", [(1, 0, 1, 16), (1, 5, 1, 1), (7, 30, 1, 16), (24, 2000, 1, 16),
                                                 (33, 100, 70, 24), (300, 40, 9, 8), (1000, 3, 2, 4), (2, 10, 4000, 32),
                                                 (8192, 2, 1, 1)])
def test_tables(batch, mean, new, page):
    rng = np.random.default_rng(batch + page)
    lens = rng.integers(0, 2 * mean + 1, batch)
    news = rng.integers(0, 2 * new, batch) if new > 1 else np.ones(batch, dtype=int)
    cols = int(-(-(lens + news).max() // page)) + 1
    need = int((-(-(lens + news) // page) - -(-lens // page)).sum())
    pages = batch * cols + need + 3
    order = rng.permutation(pages)
    table = order[:batch * cols].reshape(batch, cols)
    free = order[batch * cols:]
    # rows behind the last request, a free list that starts and ends inside its buffer, a strided table
    run_tables(lens, news, page, pages, cols, free, span=[1, len(free)], rows=int(news.sum()) + 5, table=table,
               stride=cols + 3)


def test_tables_run_out_of_pages():
    # 2 pages left for needs of 1, 0, 3, 1
    ref = run_tables([4, 3, 4, 0], [2, 1, 10, 1], 4, 20, 5, [11, 12, 13], span=[1, 3])
    assert ref[5] == bd.DEV_OUT_OF_PAGES and ref[3].tolist() == [6, 4, 8, 0]
    ref = run_tables([4, 3], [2, 1], 4, 20, 5, [11], span=[1, 1])
    assert ref[5] == bd.DEV_OUT_OF_PAGES and ref[3].tolist() == [4, 4]


@pytest.mark.parametrize("kw,status", [
    (dict(lens=[4, -1, 3], new=[2, 2, 2]), bd.DEV_BAD_LENGTH),
    (dict(lens=[4, 19, 3], new=[2, 2, 2]), bd.DEV_BAD_LENGTH),                       # would outgrow its row
    (dict(lens=[4, 2 ** 31 - 1, 3], new=[2, 2, 2]), bd.DEV_BAD_LENGTH),
    (dict(lens=[4, 4, 3], new=[2, 2, 2], cu=[0, 4, 2, 6]), bd.DEV_BAD_LENGTH),       # decreasing
    (dict(lens=[4, 4, 3], new=[2, 2, 2], cu=[-1, 2, 4, 6]), bd.DEV_BAD_LENGTH),
    (dict(lens=[4, 4, 3], new=[2, 2, 2], rows=5), bd.DEV_BAD_LENGTH),                # past the rows
    (dict(lens=[4, 4, 3], new=[2, 2, 2], span=[-1, 3]), bd.DEV_BAD_OFFSET | bd.DEV_OUT_OF_PAGES),
    (dict(lens=[4, 4, 3], new=[2, 2, 2], span=[2, 9]), bd.DEV_BAD_OFFSET | bd.DEV_OUT_OF_PAGES),
    (dict(lens=[4, 4, 3], new=[2, 2, 2], span=[3, 1]), bd.DEV_BAD_OFFSET | bd.DEV_OUT_OF_PAGES),
    (dict(lens=[4, 4, 3], new=[2, 2, 2], free=[7, 20, 8]), bd.DEV_BAD_PAGE),         # a free page that is none
    (dict(lens=[4, 4, 3], new=[2, 2, 2], free=[7, -2, 8]), bd.DEV_BAD_PAGE),
    (dict(lens=[4, 4, 3], new=[2, 2, 2], table=np.array([[0] * 5, [1] * 5, [-1] * 5])), bd.DEV_BAD_PAGE),
    (dict(lens=[4, 4, 3], new=[0, 0, 0]), 0),
    (dict(lens=[4, 4, 3], new=[0, 0, 0], rows=3), 0),
    (dict(lens=[4, 4, 3], new=[2, 2, 2], cu=[2, 4, 6, 8], rows=9), 0),               # rows before the first request
    (dict(lens=[], new=[], rows=4), 0),
])
def test_tables_of_bad_and_empty_inputs(kw, status):
    args = dict(page=4, pages=20, cols=5, free=[7, 9, 8])
    args.update(kw)
    assert run_tables(**args)[5] == status


# ---------------------------------------------------------------------- one-token attention
class Cache:
    """Requests of the given lengths over randomly placed pages; every cache row outside
    them holds NaN."""

    def __init__(self, seed, lens, h_kv, d, page, dtype, heads_first=False, cols=None, gap=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        used = [-(-n // page) for n in lens]
        self.pages = sum(used) + 4
        order = torch.randperm(self.pages, generator=torch.Generator().manual_seed(seed)).int()
        self.table = torch.full((len(lens), cols or max(used + [1])), 2 ** 30, dtype=torch.int32)
        shape = (self.pages, h_kv, page, d + gap) if heads_first else (self.pages, page, h_kv, d + gap)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=dtype, device="cuda")[..., :d] for _ in range(2))
        if heads_first:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        at = 0
        for b, n in enumerate(lens):
            held = order[at:at + used[b]]
            at += used[b]
            self.table[b, :used[b]] = held
            key = torch.arange(n, device="cuda")
            page_of = held.cuda().long()[key // page]
            for c in (self.k, self.v):
                c[page_of, key % page] = torch.randn((n, h_kv, d), generator=g, device="cuda").to(dtype)
        self.table = self.table.cuda()
        self.lens = ints(lens)
        self.gen = g


def check(cache, q, o, lse, scale=None, window=None, table=None, lens=None, o0=None, lse0=None, matrix=True):
    """Compares O and Stats [batch, h_q] with the oracle within the derived bound."""
    dtype = q.dtype
    scale = q.shape[2] ** -0.5 if scale is None else scale
    table = (cache.table if table is None else table).cpu().numpy()
    lens = (cache.lens if lens is None else lens).cpu().numpy()
    k, v, qn = f64(cache.k), f64(cache.v), f64(q)
    win = None if window is None else window.cpu().numpy()
    ref_o, ref_lse, status = paged_attention(qn, k, v, table, lens, scale, win, o0, lse0)
    got_o, got_lse = f64(o), f64(lse)
    pages, page, h_kv, _ = k.shape
    group = q.shape[1] // h_kv
    for b in range(len(lens)):
        n = int(lens[b])
        if n < 0 or n > table.shape[1] * page:
            assert np.array_equal(got_o[b], ref_o[b]) and np.array_equal(got_lse[b], ref_lse[b])
            continue
        low = max(0, n - 1 - int(win[b])) if win is not None and win[b] >= 0 else 0
        keys = np.arange(low, n)
        held = table[b, keys // page]
        keys, held = keys[(held >= 0) & (held < pages)], held[(held >= 0) & (held < pages)]
        if len(keys) == 0:
            assert (got_o[b] == 0).all() and np.isneginf(got_lse[b]).all()
            continue
        for h in range(q.shape[1]):
            kk, vv = k[held, keys % page, h // group], np.abs(v[held, keys % page, h // group])
            m = abs(scale) * (np.abs(kk) @ np.abs(qn[b, h])).max()
            e = 64 * U * m + (len(keys) / 64 + 96) * U
            p = np.exp(scale * (kk @ qn[b, h]) - ref_lse[b, h])
            rest = HALF[dtype] ** 2 if matrix else 0.0
            bound = HALF[dtype] * np.abs(ref_o[b, h]) + (rest + 2 * e) * (p @ vv)
            if matrix and dtype == torch.float16:
                bound = bound + len(keys) * 2.0 ** -25 * vv.max(0)
            if dtype == torch.float16:
                bound = bound + 2.0 ** -25
            err = np.abs(got_o[b, h] - ref_o[b, h])
            assert (err <= bound).all(), (b, h, float((err - bound).max()))
            assert abs(got_lse[b, h] - ref_lse[b, h]) <= 2 * e + 4 * U * abs(ref_lse[b, h]), (b, h)
    return status


def random_q(cache, h_q, gap=0):
    b, d = cache.lens.numel(), cache.k.shape[3]
    backing = torch.randn((b, h_q + gap, d), generator=cache.gen, device="cuda").to(cache.k.dtype)
    return backing[:, :h_q]


CASES = [
    # lens, h_q, h_kv, d, page, dtype, heads_first
    ([1], 8, 1, 128, 16, torch.bfloat16, False),
    ([0, 1, 2, 15, 16, 17, 63, 64, 65, 200], 32, 8, 128, 16, torch.bfloat16, False),
    ([700], 32, 8, 128, 16, torch.bfloat16, True),
    ([3000, 1, 0, 257], 16, 16, 64, 24, torch.float16, False),       # one query head per kv head
    ([513, 90], 10, 2, 64, 8, torch.float16, True),                  # groups of 5
    ([511, 33, 1025], 16, 1, 128, 64, torch.bfloat16, False),        # a group of 16
    ([300, 31], 14, 1, 80, 1, torch.bfloat16, False),                # groups of 14, one-row pages, d = 80
    ([400, 130], 40, 1, 128, 32, torch.float16, False),              # 40 heads: segments of 32 and 8
    ([150, 20], 72, 2, 64, 16, torch.bfloat16, True),                # 36 heads each: 32 and 4
    ([5000], 2, 1, 8, 3, torch.float16, False),
    ([777, 5], 6, 3, 40, 7, torch.bfloat16, False),
    ([1000, 0, 64], 8, 2, 128, 16, torch.float32, False),            # SIMT kernel
    ([333, 12], 9, 1, 96, 5, torch.float32, True),                   # nine heads: 8 and 1
    ([100, 70], 4, 2, 33, 6, torch.float32, False),
    ([100, 70], 4, 2, 57, 6, torch.bfloat16, False),                 # SIMT: d % 8 != 0
    ([9, 1, 1], 3, 3, 1, 4, torch.float16, False),
]


@pytest.mark.parametrize("lens,h_q,h_kv,d,page,dtype,heads_first", CASES)
def test_attention(lens, h_q, h_kv, d, page, dtype, heads_first):
    cache = Cache(len(lens) + d, lens, h_kv, d, page, dtype, heads_first)
    q = random_q(cache, h_q, gap=2)
    o_back = torch.full((len(lens), h_q + 1, d), 7.0, dtype=dtype, device="cuda")
    o = o_back[:, :h_q]
    _, stats = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens, o=o)
    plan = rva.paged_decode_plan_for_tensors(q, cache.k, cache.v, o, cache.table)
    check(cache, q, o, stats.view(len(lens), h_q), matrix=plan.kernel == bd.KERNEL_MMA)
    assert (o_back[:, h_q:] == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [[0, 0, 0, 0], [1, 63, 64, 2 ** 31 - 1], [15, -1, 16, 500], [700, 899, 900, 2]])
def test_windows(window, dtype):
    lens = [900, 900, 900, 1]
    cache = Cache(3, lens, 2, 128, 16, dtype)
    q = random_q(cache, 8)
    win = ints(window)
    o, stats = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens, window_left=win)
    check(cache, q, o, stats.view(4, 8), window=win, matrix=dtype != torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch", [31, 32, 33, 127, 129, 255, 256, 257])
def test_request_counts_around_the_search_steps(batch, dtype):
    """The first worker of every request is found by 32, 128 and 256 requests at a time."""
    lens = np.random.default_rng(batch).integers(0, 40, batch)
    lens[batch // 2:batch // 2 + 20] = 0
    cache = Cache(batch, lens.tolist(), 1, 64, 8, dtype, cols=6)
    q = random_q(cache, 2)
    o, stats = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens)
    check(cache, q, o, stats.view(batch, 2), matrix=dtype != torch.float32)


def test_views_of_other_layouts():
    """Caches inside larger buffers, K and V of different strides, and an O whose odd strides
    only the SIMT kernel takes."""
    lens = [130, 47, 300]
    cache = Cache(21, lens, 2, 128, 16, torch.bfloat16)
    q = random_q(cache, 8)
    ref = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens)
    both = torch.full((cache.pages, 3, 16, 2, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    k, v = both[:, 1, :, :, 128:], torch.full((cache.pages, 2, 16, 128), float("nan"), dtype=torch.bfloat16,
                                              device="cuda").transpose(1, 2)
    k.copy_(cache.k)
    v.copy_(cache.v)
    got = rva.thd_paged_attention(q, k, v, cache.table, cache.lens)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    for gap in (1, 129):
        o = torch.zeros((3, 8, 128 + gap), dtype=torch.bfloat16, device="cuda")[..., :128]
        rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens, o=o, stats=ref[1])
        check(cache, q, o, ref[1].view(3, 8), matrix=False)


def test_odd_page_sizes_and_partly_visible_chunks():
    """Every page size at which rows of a chunk lie in one page, in several, or in pages of their
    own, with windows that begin and end inside a chunk."""
    for page in (1, 2, 3, 8, 12, 24, 40, 257):
        for dtype, d in ((torch.float16, 64), (torch.bfloat16, 128), (torch.bfloat16, 88), (torch.float32, 100)):
            cache = Cache(page + d, [200, 77, 129, 8], 2, d, page, dtype)
            q = random_q(cache, 6)
            win = ints([-1, 50, 100, 3])
            o, stats = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens, window_left=win)
            check(cache, q, o, stats.view(4, 6), window=win, matrix=dtype != torch.float32)


def test_an_empty_cache_and_no_requests():
    """No page at all: every key is in a bad page. No request: nothing happens, status 0."""
    for dtype in (torch.bfloat16, torch.float32):
        k = torch.zeros((0, 16, 2, 64), dtype=dtype, device="cuda")
        q = torch.ones((2, 4, 64), dtype=dtype, device="cuda")
        table, lens = ints([[0, 1], [5, -1]]), ints([20, 3])
        o, stats = torch.full_like(q, 7), torch.zeros(8, device="cuda")
        plan = rva.paged_decode_plan_for_tensors(q, k, k, o, table)
        ws = rva.alloc_workspace(plan, "cuda")
        rva.thd_paged_decode(plan, q, k, k, table, lens, None, o, stats, ws)
        assert rva.thd_attn_read_status(plan, ws) == bd.DEV_BAD_PAGE
        assert (o == 0).all() and (stats == float("-inf")).all()
        none = rva.thd_paged_attention(q[:0], k, k, table[:0], lens[:0])
        assert none[0].shape == (0, 4, 64)


def test_many_requests_most_of_them_empty():
    rng = np.random.default_rng(8)
    lens = np.where(rng.random(700) < 0.8, 0, rng.integers(1, 90, 700))
    lens[:100] = 0
    lens[-40:] = 0
    cache = Cache(4, lens.tolist(), 2, 64, 16, torch.bfloat16, cols=8)
    q = random_q(cache, 4)
    o, stats = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens)
    check(cache, q, o, stats.view(700, 4))
    empty = cache.lens * 0
    o.fill_(3)
    rva.thd_paged_attention(q, cache.k, cache.v, cache.table, empty, o=o, stats=stats)
    assert (o == 0).all() and (stats == float("-inf")).all()


@pytest.mark.parametrize("h_q,h_kv", [(8, 1), (32, 8)])
def test_long_requests_cross_many_ctas(h_q, h_kv):
    cache = Cache(5, [40000, 3, 23456], h_kv, 128, 16, torch.bfloat16)
    q = random_q(cache, h_q)
    o, stats = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens)
    check(cache, q, o, stats.view(3, h_q))


@pytest.mark.parametrize("kernel", [bd.KERNEL_MMA, bd.KERNEL_SIMT])
def test_bad_lengths_and_pages(kernel):
    lens = [100, 50, 60, 70, 33]
    cache = Cache(6, lens, 2, 64, 16, torch.bfloat16, cols=7)
    q = random_q(cache, 8)
    table, bad = cache.table.clone(), cache.lens.clone()
    table[0, 3] = -1                    # keys 48 .. 63 count as not visible
    table[2, :4] = cache.pages          # every page of request 2
    table[3, 1] = -2 ** 31
    bad[1], bad[4] = -1, 7 * 16 + 1     # rows stay as they are
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    stats = torch.full((5 * 8,), 5.0, device="cuda")
    plan = rva.paged_decode_plan_for_tensors(q, cache.k, cache.v, o, table, kernel=kernel)
    ws = torch.full((plan.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")
    rva.thd_paged_decode(plan, q, cache.k, cache.v, table, bad, None, o, stats, ws)
    assert rva.thd_attn_read_status(plan, ws) == bd.DEV_BAD_LENGTH | bd.DEV_BAD_PAGE
    check(cache, q, o, stats.view(5, 8), table=table, lens=bad, o0=np.full(q.shape, 7.0), lse0=np.full((5, 8), 5.0),
          matrix=kernel == bd.KERNEL_MMA)
    rva.thd_paged_decode(plan, q, cache.k, cache.v, cache.table, cache.lens, None, o, None, ws)
    assert rva.thd_attn_read_status(plan, ws) == 0
    check(cache, q, o, rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens)[1].view(5, 8))


def test_stats_layouts_scales_and_shared_pages():
    cache = Cache(7, [90, 40, 130], 2, 128, 16, torch.float16)
    cache.table[1] = cache.table[2]     # request 1 reads the beginning of request 2's pages
    q = random_q(cache, 6)
    for layout in (bd.STATS_TOKEN_MAJOR, bd.STATS_HEAD_MAJOR):
        for scale in (None, 0.0, -0.05, 0.7):
            o, stats = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens, stats_layout=layout,
                                               softmax_scale=scale)
            check(cache, q, o, stats.view(3, 6) if layout == bd.STATS_TOKEN_MAJOR else stats.view(6, 3).t(), scale=scale)


def test_large_scores_and_infinite_values():
    """Scores far apart (one key takes all), and an infinite V row, which is the answer where it
    is seen and nothing where it is masked."""
    cache = Cache(8, [200], 1, 64, 16, torch.float32)
    q = random_q(cache, 4) * 40
    o, stats = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens, softmax_scale=1.0)
    check(cache, q, o, stats.view(1, 4), scale=1.0, matrix=False)
    cache = Cache(8, [200], 1, 64, 16, torch.bfloat16)
    q = random_q(cache, 4)
    page, row = int(cache.table[0, 100 // 16]), 100 % 16
    cache.v[page, row] = float("inf")
    o, _ = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens)
    assert (o == float("inf")).all()
    o, _ = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens, window_left=ints([98]))
    assert torch.isfinite(o).all()
    cache.k[page, row] = float("nan")
    o, _ = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens)
    assert o.isnan().all()
    o, stats = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens, window_left=ints([98]))
    assert torch.isfinite(o).all() and torch.isfinite(stats).all()


def test_matrix_and_simt_kernels_agree():
    cache = Cache(9, [1200, 77, 0, 5], 4, 128, 16, torch.float16)
    q = random_q(cache, 20)
    a, b = (rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens, kernel=k)
            for k in (bd.KERNEL_MMA, bd.KERNEL_SIMT))
    check(cache, q, a[0], a[1].view(4, 20))
    check(cache, q, b[0], b[1].view(4, 20), matrix=False)


def test_equal_bits_and_a_captured_call_follows_its_inputs():
    cache = Cache(10, [2000, 700, 0, 33], 4, 128, 16, torch.bfloat16)
    q = random_q(cache, 16)
    a, b = (rva.thd_paged_attention(q, cache.k, cache.v, cache.table, cache.lens) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    lens, graph = cache.lens.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, lens)
    for new in ([2000, 700, 0, 33], [1, 699, 0, 20], [0, 0, 0, 0], [1999, 64, 0, 1]):
        lens.copy_(ints(new))
        graph.replay()
        ref = rva.thd_paged_attention(q, cache.k, cache.v, cache.table, ints(new))
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_two_calls_at_once_on_two_streams():
    caches = [Cache(11 + i, [3000, 100], 2, 128, 16, torch.bfloat16) for i in range(2)]
    qs = [random_q(c, 16) for c in caches]
    refs = [rva.thd_paged_attention(q, c.k, c.v, c.table, c.lens) for q, c in zip(qs, caches)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got = [rva.thd_paged_attention(q, c.k, c.v, c.table, c.lens, stream=s) for q, c, s in zip(qs, caches, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, refs):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_guard_bands():
    """Workspace, O and Stats between bytes that have to survive."""
    cache = Cache(12, [900, 64, 1], 2, 128, 16, torch.bfloat16)
    q = random_q(cache, 40)
    o_plan = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    plan = rva.paged_decode_plan_for_tensors(q, cache.k, cache.v, o_plan, cache.table)

    def banded(n):
        whole = torch.full((n + 2 * 65536,), 0x5A, dtype=torch.uint8, device="cuda")
        return whole, whole[65536:65536 + n]

    (wa, ws), (oa, ob), (sa, sb) = banded(plan.workspace_bytes), banded(q.numel() * 2), banded(3 * 40 * 4)
    o, stats = ob.view(torch.bfloat16).view(q.shape), sb.view(torch.float32)
    rva.thd_paged_decode(plan, q, cache.k, cache.v, cache.table, cache.lens, None, o, stats, ws)
    torch.cuda.synchronize()
    for whole, n in ((wa, plan.workspace_bytes), (oa, q.numel() * 2), (sa, 3 * 40 * 4)):
        assert (whole[:65536] == 0x5A).all() and (whole[65536 + n:] == 0x5A).all()
    check(cache, q, o, stats.view(3, 40))


def test_pages_past_32_bits_of_elements():
    """A cache of more than 2^32 elements, whose last pages are read."""
    page, h_kv, d = 16, 8, 128
    pages = (1 << 32) // (page * h_kv * d) + 5
    k, v = (torch.empty((pages, page, h_kv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    small = Cache(13, [60], h_kv, d, page, torch.bfloat16)
    table = torch.tensor([[pages - 1, pages - 4, 0, pages - 2]], dtype=torch.int32, device="cuda")
    for big, c in ((k, small.k), (v, small.v)):
        big[table[0].long()] = c[small.table[0].long()]
    q = random_q(small, 32)
    a = rva.thd_paged_attention(q, small.k, small.v, small.table, small.lens)
    b = rva.thd_paged_attention(q, k, v, table, small.lens)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------------- the serving step
@pytest.mark.parametrize("dtype,h_q,h_kv,d,page", [(torch.bfloat16, 16, 4, 128, 16), (torch.float16, 6, 6, 64, 24),
                                                   (torch.float32, 4, 2, 96, 5)])
def test_serving_steps(dtype, h_q, h_kv, d, page):
    """Prefill and four decode steps of three requests, table -> norm, rotation and cache ->
    attention, without a host read in between; each step's O against the oracle over the keys
    that the plain formula gives for all tokens so far."""
    batch, cols, pages, max_pos = 3, 12, 40, 400
    g = torch.Generator(device="cuda").manual_seed(d)
    half = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    table = torch.cat([half.cos(), half.sin()], 1).float().cuda()
    w_q, w_k = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype) for _ in range(2))
    k_cache, v_cache = (torch.full((pages, page, h_kv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    bt = torch.full((batch, cols), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).int().cuda()
    lens, span = ints([0, 0, 0]), ints([0, pages])
    keys = [torch.zeros((0, h_kv, d), dtype=torch.float64) for _ in range(batch)]
    vals = [torch.zeros((0, h_kv, d), dtype=torch.float64) for _ in range(batch)]
    for news in ([20, 1, 37], [1, 1, 1], [1, 0, 1], [1, 1, 1], [1, 1, 1]):
        rows = 64 if max(news) > 1 else 4      # pad rows behind the last request
        cu = ints(np.concatenate([[0], np.cumsum(news)]).tolist())
        slots, pos, lens_out, begin = rva.thd_paged_extend(lens, cu, free, span, bt, page_size=page, num_pages=pages,
                                                           rows=rows)
        qkv = torch.randn((rows, h_q + 2 * h_kv, d), generator=g, device="cuda").to(dtype)
        q, k, v = qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:]
        qz = rva.thd_qk_norm_rope_append(q, k, v, w_q, w_k, table, pos, slots, k_cache, v_cache)
        last = (cu[1:] - 1).clamp(min=0).long()
        o, stats = rva.thd_paged_attention(qz[last], k_cache, v_cache, bt, lens_out)
        # the oracle
        at = 0
        for b, n in enumerate(news):
            p = np.arange(len(keys[b]), len(keys[b]) + n)
            kz = norm_rope_fwd(f64(k)[at:at + n], f64(w_k), f64(table), p, 1e-6, False, np.zeros((n, h_kv, d)))
            keys[b] = torch.cat([keys[b], torch.from_numpy(kz)])
            vals[b] = torch.cat([vals[b], torch.from_numpy(f64(v)[at:at + n])])
            at += n
            if n == 0:
                continue
            qr = norm_rope_fwd(f64(q)[at - 1:at], f64(w_q), f64(table), p[-1:], 1e-6, False, np.zeros((1, h_q, d)))[0]
            for h in range(h_q):
                kk, vv = keys[b][:, h // (h_q // h_kv)].numpy(), vals[b][:, h // (h_q // h_kv)].numpy()
                s = kk @ qr[h] * d ** -0.5
                m = (np.abs(kk) @ np.abs(qr[h])).max() * d ** -0.5
                prob = np.exp(s - s.max())
                prob /= prob.sum()
                # Q and K are rounded to the storage type in between: their scores by 2 h M more
                e = 3 * HALF[dtype] * m + (64 * m + 100) * U
                bound = HALF[dtype] * np.abs(prob @ vv) + (HALF[dtype] + 2 * e) * (prob @ np.abs(vv)) + 64 * 2.0 ** -25
                assert (np.abs(f64(o)[b, h] - prob @ vv) <= bound).all(), (news, b, h)
        assert lens_out.tolist() == [len(x) for x in keys]
        lens, span = lens_out, torch.cat([begin, span[1:]])
    assert not torch.isnan(o).any()


def test_a_captured_serving_step_replays():
    """The three calls of a decode step as one CUDA graph, lengths and free pages fed back on
    the device between replays; against the same steps made call by call."""
    batch, h_q, h_kv, d, page, pages, cols = 4, 8, 2, 64, 4, 64, 16
    dtype, max_pos = torch.bfloat16, 100

    def fresh():
        g = torch.Generator(device="cuda").manual_seed(6)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
        half = torch.arange(max_pos)[:, None] * 10000.0 ** (-torch.arange(0, d, 2) / d)
        return dict(qkv=rand(batch, h_q + 2 * h_kv, d), w=rand(d), table=torch.cat([half.cos(), half.sin()], 1).cuda(),
                    k=rand(pages, page, h_kv, d), v=rand(pages, page, h_kv, d),
                    bt=torch.arange(batch * cols, dtype=torch.int32, device="cuda").view(batch, cols) % 13,
                    free=torch.arange(20, 60, dtype=torch.int32, device="cuda"), lens=ints([3, 4, 0, 9]), span=ints([0, 40]),
                    cu=ints([0, 1, 2, 3, 4]))

    def step(s):
        q, k, v = s["qkv"][:, :h_q], s["qkv"][:, h_q:h_q + h_kv], s["qkv"][:, h_q + h_kv:]
        slots, pos, lens, begin = rva.thd_paged_extend(s["lens"], s["cu"], s["free"], s["span"], s["bt"], page_size=page,
                                                       num_pages=pages, rows=batch)
        qz = rva.thd_qk_norm_rope_append(q, k, v, s["w"], s["w"], s["table"], pos, slots, s["k"], s["v"])
        o, stats = rva.thd_paged_attention(qz, s["k"], s["v"], s["bt"], lens)
        s["lens"].copy_(lens)
        s["span"][:1].copy_(begin)
        s["qkv"].mul_(-0.75)
        return o

    a, b = fresh(), fresh()
    step(a)
    step(b)        # plans and modules exist before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(b)
    for _ in range(6):
        ref = step(a)
        graph.replay()
        assert torch.equal(ref, out) and torch.equal(a["lens"], b["lens"]) and torch.equal(a["bt"], b["bt"])
        assert torch.equal(a["k"], b["k"]) and torch.equal(a["v"], b["v"])
