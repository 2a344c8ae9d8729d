"""CPU oracles of the paged cache: page tables of a step (plain Python, one token at a
time) and one-token attention (float64 numpy, one request and head at a time)."""
from __future__ import annotations

import numpy as np

BAD_LENGTH, BAD_OFFSET, BAD_PAGE, OUT_OF_PAGES = 1, 2, 64, 128


def paged_tables(seq_lens, cu_new, free_pages, free_span, block_table, page_size, num_pages, rows):
    """Returns (block_table, slot_map, positions, seq_lens_out, free_begin_out, status)."""
    table = np.array(block_table, dtype=np.int64)
    batch, max_pages = table.shape
    slots, positions = [-1] * rows, [-1] * rows
    lens_out = [int(n) for n in seq_lens]
    begin, end = (int(v) for v in free_span)
    status = 0
    if begin < 0 or end < begin or end > len(free_pages):
        status |= BAD_OFFSET
        end = begin
    ordered = all(0 <= cu_new[b] <= cu_new[b + 1] <= rows for b in range(batch))
    if not ordered:
        return table, np.array(slots), np.array(positions), np.array(lens_out), begin, status | BAD_LENGTH
    at = begin
    for b in range(batch):
        n, new = int(seq_lens[b]), int(cu_new[b + 1] - cu_new[b])
        if n < 0 or n + new > max_pages * page_size:
            status |= BAD_LENGTH
            continue
        held = -(-n // page_size)   # pages, those granted in this step among them
        served = 0
        for t in range(new):
            pos = n + t
            column, row = divmod(pos, page_size)
            if column >= -(-n // page_size) and row == 0:   # the first token of a new page
                if at < end:
                    page = int(free_pages[at])
                    at += 1
                    held += 1
                    if not 0 <= page < num_pages:
                        page = -1
                        status |= BAD_PAGE
                else:
                    page = -1
                    status |= OUT_OF_PAGES
                table[b, column] = page
            page = int(table[b, column])
            if column < -(-n // page_size) and not 0 <= page < num_pages:
                page = -1
                status |= BAD_PAGE
            positions[cu_new[b] + t] = pos
            slots[cu_new[b] + t] = page * page_size + row if page >= 0 else -1
            served += pos < held * page_size
        lens_out[b] = n + served
    return table, np.array(slots), np.array(positions), np.array(lens_out), at, status


def paged_attention(q, k_cache, v_cache, block_table, seq_lens, scale, window_left=None, o=None, lse=None):
    """q [batch, h_q, d]; caches [pages, page_size, h_kv, d]. Returns (o, lse [batch, h_q],
    status); rows of an invalid length keep the given o and lse."""
    q = np.asarray(q, dtype=np.float64)
    batch, h_q, d = q.shape
    pages, page_size, h_kv, _ = k_cache.shape
    o = np.zeros_like(q) if o is None else np.array(o, dtype=np.float64)
    lse = np.zeros((batch, h_q)) if lse is None else np.array(lse, dtype=np.float64)
    status = 0
    for b in range(batch):
        n = int(seq_lens[b])
        if n < 0 or n > block_table.shape[1] * page_size:
            status |= BAD_LENGTH
            continue
        w = -1 if window_left is None else int(window_left[b])
        keys = np.arange(max(0, n - 1 - w) if w >= 0 else 0, n)
        held = np.asarray(block_table)[b, keys // page_size]
        good = (held >= 0) & (held < pages)
        if not good.all():
            status |= BAD_PAGE
        keys, held = keys[good], held[good]
        for h in range(h_q):
            g = h // (h_q // h_kv)
            s = scale * (np.asarray(k_cache[held, keys % page_size, g], dtype=np.float64) @ q[b, h])
            if len(s) == 0:
                o[b, h], lse[b, h] = 0.0, -np.inf
                continue
            top = s.max()
            e = np.exp(s - top)
            lse[b, h] = top + np.log(e.sum())
            o[b, h] = (e / e.sum()) @ np.asarray(v_cache[held, keys % page_size, g], dtype=np.float64)
    return o, lse, status
