"""fp64 / integer CPU oracle of the dense paged path: the page pool with its block tables and
slot maps, the write of new rows, and the attention of one new token over a whole cache.

Test infrastructure only; nothing of the library runs here.
"""
from __future__ import annotations

import numpy as np

PAGE = 16
DEVERR_PAGE_RANGE, DEVERR_LENGTH, DEVERR_NO_PAGES = 0x1, 0x2, 0x8


def _pages(n):
    return -(-n // PAGE)


class Pool:
    """Free pages as a stack, taken from its end."""

    def __init__(self, num_pages, free=None):
        self.num_pages = num_pages
        self.free = list(range(num_pages)) if free is None else list(free)


def extend(pool, table, lens, new, max_new):
    """(table, lens after, token_start, slot_map, positions, error bits) after new[b] tokens behind lens[b];
    takes its pages from ``pool``. ``table``: int array [B][width] (copied)."""
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    err, start, exhausted = 0, [0], False
    slots = np.full(max_new, -1, dtype=np.int64)
    pos = np.zeros(max_new, dtype=np.int64)
    after = []
    at = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        first, at = at, at + max(m, 0)
        start.append(min(at, max_new))
        after.append(n)
        if n < 0 or m < 0 or n + m > width * PAGE or at > max_new:
            err |= DEVERR_LENGTH
            continue
        need = _pages(n + m) - _pages(n)
        if need and (exhausted or need > len(pool.free)):
            exhausted = True
            err |= DEVERR_NO_PAGES
            continue
        for p in range(_pages(n), _pages(n + m)):
            page = pool.free.pop()
            if not 0 <= page < pool.num_pages:
                err |= DEVERR_PAGE_RANGE
                page = -1
            table[b, p] = page
        for i in range(m):
            j = n + i
            page = table[b, j // PAGE]
            pos[first + i] = j
            if 0 <= page < pool.num_pages:
                slots[first + i] = page * PAGE + j % PAGE
            else:
                err |= DEVERR_PAGE_RANGE
        after[b] = n + m
    return table, after, start, slots, pos, err


def release(pool, table, lens, keep=None):
    """Pushes the pages of the tokens behind keep[b] back onto ``pool``; returns the error bits."""
    err, back = 0, []
    for b, n in enumerate(lens):
        k = 0 if keep is None else keep[b]
        if k < 0 or k > n or n > table.shape[1] * PAGE:
            err |= DEVERR_LENGTH
            continue
        back += [int(table[b, p]) for p in range(_pages(k), _pages(n))]
    if len(pool.free) + len(back) > pool.num_pages:
        return err | DEVERR_PAGE_RANGE
    for page in reversed(back):
        if not 0 <= page < pool.num_pages:
            err |= DEVERR_PAGE_RANGE
            page = -1
        pool.free.append(page)
    return err


def store(k, v, summary, k_new, v_new, slots):
    """Rows into their slots in token order, and the bounds of the pages they touch. Arrays [P][H][16][D]
    (summary [P][H][2][D] or None), changed in place."""
    fresh = {int(s) // PAGE for s in slots if s >= 0 and s % PAGE == 0 and s < k.shape[0] * PAGE}
    begun = set()
    for t, s in enumerate(slots):
        if s < 0 or s >= k.shape[0] * PAGE:
            continue
        p, i = int(s) // PAGE, int(s) % PAGE
        k[p, :, i] = k_new[t]
        if v is not None and v_new is not None:
            v[p, :, i] = v_new[t]
        if summary is not None:
            if p in fresh and p not in begun:
                summary[p, :, 0], summary[p, :, 1] = k_new[t], k_new[t]
            else:
                summary[p, :, 0] = np.minimum(summary[p, :, 0], k_new[t])
                summary[p, :, 1] = np.maximum(summary[p, :, 1], k_new[t])
            begun.add(p)


def kept_positions(n, sink, recent):
    """Positions that the query sees, ascending."""
    if recent <= 0:
        return np.arange(n)
    j = np.arange(n)
    return j[(j < sink) | (j >= n - recent)]


def decode(k, v, table, lens, q, sm_scale, dv, sink=0, recent=0):
    """out [B][Hq][dv], lse [B][Hq] in fp64 and, for the tests' error bounds, the weighted magnitudes
    sum_j softmax(z)_j |v_j| and the largest sm_scale * sum_c |q_c k_jc| of each row. Numpy arrays; v None: the
    value is the key row's first dv dims."""
    B, Hq = q.shape[:2]
    H = k.shape[1]
    G = Hq // H
    out = np.zeros((B, Hq, dv))
    mag = np.zeros((B, Hq, dv))
    lse = np.full((B, Hq), -np.inf)
    zmag = np.zeros((B, Hq))
    for b in range(B):
        j = kept_positions(int(lens[b]), sink, recent)
        if not len(j):
            continue
        page = table[b, j // PAGE]
        for h in range(H):
            keys = k[page, h, j % PAGE].astype(np.float64)
            vals = keys[:, :dv] if v is None else v[page, h, j % PAGE].astype(np.float64)
            for a in range(h * G, (h + 1) * G):
                qa = q[b, a].astype(np.float64)
                z = sm_scale * (keys @ qa)
                m = z.max()
                e = np.exp(z - m)
                lse[b, a] = m + np.log(e.sum())
                w = e / e.sum()
                out[b, a] = w @ vals
                mag[b, a] = w @ np.abs(vals)
                zmag[b, a] = abs(sm_scale) * (np.abs(keys) @ np.abs(qa)).max()
    return out, lse, mag, zmag
