"""Paged key-value cache and tree attention oracle (test infrastructure only).

Plain float64 / integer numpy, one request at a time, from the definitions:

* ``pages_resize``   -- block tables from lengths over one free list: returns
  first (in request and column order, the first one on top), then takes from the
  top in request order until one does not fit.
* ``tree_slots``     -- slot = table[t // P] * P + t % P and position = ctx + depth.
* ``append``         -- rows into slots.
* ``tree_attention`` -- softmax(scale q K^T) V over the tokens a row sees: the
  context, and the nodes j <= i whose mask bit is set (DSpark explainer
  (xiaohu-jiedu), one round from drafting to confirmation: the target reads the
  whole draft in one forward).
* ``commit``         -- the accepted path's rows moved behind the root.

Parity status: ``tree_attention`` is pinned by attention over each node's own
root path as a plain sequence; ``pages_resize`` by page conservation and by
growing and shrinking back; ``tree_slots``, ``append`` and ``commit`` by reading
the cache back as sequences (``tests/test_oracle_kvcache.py``).
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

BAD_COUNT, BAD_PAGE, NO_PAGE, BAD_LENGTH, BAD_PATH = 4, 64, 128, 256, 512


def pages_resize(length, table, held, free, page_size, n_pages):
    """(table, held, free list, status) after the resize; inputs are not changed.
    free: the list of free pages, its top last."""
    table, held, free = np.array(table), np.array(held), [int(x) for x in free]
    batch, width = table.shape
    status = np.zeros(batch, np.int32)
    want = [-(-int(t) // page_size) for t in length]
    back = []
    for b in range(batch):
        if length[b] < 0 or want[b] > width or not 0 <= held[b] <= width:
            status[b] = BAD_LENGTH
            continue
        if want[b] < held[b]:
            pages = [int(x) for x in table[b, want[b]:held[b]]]
            if any(not 0 <= p < n_pages for p in pages):
                status[b] = BAD_PAGE
                continue
            back += pages
            table[b, want[b]:held[b]] = -1
            held[b] = want[b]
    free += back[::-1]
    short = False
    for b in range(batch):
        if status[b] or want[b] <= held[b]:
            continue
        need = want[b] - int(held[b])
        short = short or need > len(free)
        if short:
            status[b] = NO_PAGE
            continue
        for c in range(held[b], want[b]):
            table[b, c] = free.pop()
        held[b] = want[b]
    return table, held, free, status


def tree_slots(ctx, count, depth, table, n_stride, page_size, n_pages):
    batch, width = np.shape(table)
    slot = np.full((batch, n_stride), -1, np.int64)
    pos = np.full((batch, n_stride), -1, np.int64)
    status = np.zeros(batch, np.int32)
    for b in range(batch):
        if not 0 <= count[b] <= n_stride:
            status[b] |= BAD_COUNT
        if ctx[b] < 0 or (not status[b] and ctx[b] + count[b] > width * page_size):
            status[b] |= BAD_LENGTH
        if status[b]:
            continue
        for i in range(int(count[b])):
            t = int(ctx[b]) + i
            page = int(table[b][t // page_size])
            if 0 <= page < n_pages:
                slot[b, i] = page * page_size + t % page_size
            else:
                status[b] = BAD_PAGE
            pos[b, i] = int(ctx[b]) + (i if depth is None else int(depth[b][i]))
    return slot, pos, status


def append(k_new, v_new, slot, k, v):
    """(k, v, status) with caches [n_pages][page_size][heads][d]; inputs are not changed."""
    k, v = np.array(k), np.array(v)
    page = k.shape[1]
    status = np.zeros(len(slot), np.int32)
    for b in range(len(slot)):
        for i, s in enumerate(slot[b]):
            if s >= k.shape[0] * page:
                status[b] = BAD_PAGE
            elif s >= 0:
                k[s // page, s % page], v[s // page, s % page] = k_new[b][i], v_new[b][i]
    return k, v, status


@dataclass
class AttnResult:
    out: np.ndarray       # [batch][n][heads_q][d] float64
    lse: np.ndarray       # [batch][n][heads_q]
    weight: np.ndarray    # like out: sum softmax_t |v_t|, for error bounds
    size: np.ndarray      # like lse: max_t scale sum |q| |k_t|, for error bounds
    status: np.ndarray


def sees(mask_row, i, j) -> bool:
    return j <= i and (mask_row is None or bool((int(mask_row[j // 32]) >> (j % 32)) & 1))


def tree_attention(q, k, v, table, ctx, count, mask, scale) -> AttnResult:
    """q [batch][n][hq][d], caches [n_pages][page_size][hkv][d], all float64; mask uint32
    words or None."""
    batch, n, hq, d = q.shape
    n_pages, page, hkv, _ = k.shape
    g = hq // hkv
    width = np.shape(table)[1]
    out, weight = np.zeros(q.shape), np.zeros(q.shape)
    lse, size = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    status = np.zeros(batch, np.int32)
    for b in range(batch):
        c, m = int(ctx[b]), int(count[b])
        if not 0 <= m <= n:
            status[b] |= BAD_COUNT
        if c < 0 or (not status[b] and c + m > width * page):
            status[b] |= BAD_LENGTH
        if status[b]:
            continue
        t = np.arange(c + m)
        pages = np.asarray(table[b])[t // page] if m else np.zeros(0, int)
        t = t[: len(pages)]
        here = (pages >= 0) & (pages < n_pages)
        if m and not here.all():
            status[b] |= BAD_PAGE
        for i in range(m):
            vis = np.array([tt < c or sees(None if mask is None else mask[b][i], i, tt - c) for tt in t])
            vis &= here
            if not vis.any():
                continue
            kk, vv = k[pages[vis], t[vis] % page], v[pages[vis], t[vis] % page]
            for h in range(hq):
                s = scale * (kk[:, h // g] @ q[b, i, h])
                mx = s.max()
                e = np.exp(s - mx)
                p = e / e.sum()
                out[b, i, h] = p @ vv[:, h // g]
                weight[b, i, h] = p @ np.abs(vv[:, h // g])
                lse[b, i, h] = mx + np.log(e.sum())
                size[b, i, h] = abs(scale) * (np.abs(kk[:, h // g]) @ np.abs(q[b, i, h])).max()
    return AttnResult(out, lse, weight, size, status)


def commit(k, v, table, ctx, count, accept_len, accept_path, n_pages=None):
    """(k, v, new_len, status): caches [layers][n_pages][page_size][heads][d]; inputs are not
    changed; rows behind the new length keep their old values here."""
    old_k, old_v = k, v
    k, v = np.array(k), np.array(v)
    page, n_pages = k.shape[2], k.shape[1]
    batch, width = np.shape(table)
    new_len, status = np.array(ctx, np.int64), np.zeros(batch, np.int32)
    for b in range(batch):
        c, m, a = int(ctx[b]), int(count[b]), int(accept_len[b])
        if m < 1:
            status[b] = BAD_COUNT
        elif c < 0 or c + m > width * page:
            status[b] = BAD_LENGTH
        if not 0 <= a <= np.shape(accept_path)[1]:
            status[b] |= BAD_PATH
        if status[b]:
            continue
        path = [int(x) for x in accept_path[b][:a]]
        if any(p <= q or p >= m for p, q in zip(path, [0] + path)):
            status[b] = BAD_PATH
            continue
        where = lambda t: (int(table[b][t // page]), t % page)   # noqa: E731
        moves = [(where(c + p), where(c + 1 + i)) for i, p in enumerate(path)]
        if any(not 0 <= x[0] < n_pages for mv in moves for x in mv):
            status[b] = BAD_PAGE
            continue
        for (sp, so), (dp, do) in moves:
            k[:, dp, do], v[:, dp, do] = old_k[:, sp, so], old_v[:, sp, so]
        new_len[b] = c + 1 + a
    return k, v, new_len, status
