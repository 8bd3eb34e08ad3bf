"""Plain fp64 oracle of the paged-cache calls (see include/kvtc.h): block
tables and slot maps, the write of rows, key bounds per page, the selection of
pages, and attention of one new token. numpy, one request at a time, written
from the formulas; test infrastructure only.

Pages are float64 arrays [n_blocks, block_size, heads, head_dim] that hold the
stored values; status words are 0 or the kvtc_status a request gets.
"""
from __future__ import annotations

import math

import numpy as np

INVALID, CAPACITY = -1, -2


def n_pages(tokens: int, bs: int) -> int:
    return -(-tokens // bs)


def tables(old, new, bs, free, free_from, n_blocks, table, width, n_slots):
    """-> (table, slots, starts, taken, status); `table` [n, stride] is not changed."""
    table = np.array(table)
    slots = np.full(n_slots, -1, np.int64)
    starts, status = [0], []
    taken, at = 0, max(int(free_from), 0)
    for i, (a, b) in enumerate(zip(map(int, old), map(int, new))):
        if a < 0 or b < a or b > width * bs:
            starts.append(starts[-1])
            status.append(INVALID)
            continue
        need = n_pages(b, bs) - n_pages(a, bs)
        first = starts[-1]
        starts.append(first + b - a)
        st = 0
        if starts[-1] > n_slots or (need and at + need > len(free)):
            st = CAPACITY
        else:
            for k in range(need):
                table[i, n_pages(a, bs) + k] = free[at + k]
            taken += need
            for p in range(a, b):
                page = int(table[i, p // bs])
                if 0 <= page < n_blocks:
                    slots[first + p - a] = page * bs + p % bs
                else:
                    st = INVALID
        at += need      # a request behind one that was refused for want of pages sees its need too
        status.append(st)
    return table, slots, np.array(starts), taken, np.array(status)


def live_tokens(table_row, length, bs, n_blocks, width, blocks=None):
    """[(page, offset)] of the tokens attended to, and the status."""
    if length < 0 or length > width * bs:
        return [], INVALID
    order = range(n_pages(length, bs)) if blocks is None else [int(j) for j in blocks if 0 <= j < n_pages(length, bs)]
    found, st = [], 0
    for j in order:
        page = int(table_row[j])
        if not 0 <= page < n_blocks:
            st = INVALID
            continue
        found += [(page, t) for t in range(min(bs, length - j * bs))]
    return found, st


def bounds(k, table, lens, width, from_lens=None):
    """-> ({page: (lo, hi)}, status): the bounds that are written."""
    n_blocks, bs = k.shape[:2]
    res, status = {}, []
    for i, length in enumerate(map(int, lens)):
        st = 0
        if length < 0 or length > width * bs:
            status.append(INVALID)
            continue
        a = max(int(from_lens[i]), 0) // bs if from_lens is not None else 0
        for j in range(a, n_pages(length, bs)):
            page = int(table[i, j])
            if not 0 <= page < n_blocks:
                st = INVALID
                continue
            rows = k[page, :min(bs, length - j * bs)].reshape(-1, k.shape[2] * k.shape[3])
            res[page] = (rows.min(0), rows.max(0))       # numpy's min and max pass a NaN on
        status.append(st)
    return res, np.array(status)


def scores(q, lo, hi):
    """q [G, D], lo and hi [D] -> the score of a page, in fp64 rounded to fp32."""
    up = np.where(q < 0, 0.0, q).sum(0)
    down = np.where(q > 0, 0.0, q).sum(0)
    with np.errstate(invalid="ignore", over="ignore"):
        return np.float32(np.sum(up * hi + down * lo))


def select(q, bnd, table, lens, bs, n_blocks, width, heads, budget, first, last):
    """q [n, Hq, D], bnd [n_blocks, 2, heads, D] -> (blocks [n, heads, budget], status)."""
    n, hq, _ = q.shape
    g = hq // heads
    res = np.full((n, heads, budget), -1, np.int64)
    status = np.zeros(n, np.int64)
    for i, length in enumerate(map(int, lens)):
        if length < 0 or length > width * bs:
            status[i] = INVALID
            continue
        m = n_pages(length, bs)
        for h in range(heads):
            ranked = []
            for j in range(m):
                page = int(table[i, j])
                if not 0 <= page < n_blocks:
                    status[i] = INVALID
                    continue
                s = float(scores(q[i, h * g:(h + 1) * g], bnd[page, 0, h], bnd[page, 1, h]))
                level = 2 if j < first or j >= m - last else 1 if math.isnan(s) else 0
                ranked.append((-level, 0.0 if level else -s, j))
            keep = sorted(j for _, _, j in sorted(ranked)[:budget])
            res[i, h, :len(keep)] = keep
    return res, status


def attend(q, k, v, table, lens, width, scale, blocks=None):
    """q [n, Hq, D] -> (out [n, Hq, D], lse [n, Hq], status, slack): slack holds, per (request, query
    head), the largest scale * sum_d |q_d k_d| over the tokens, sum_t p_t |v_t| [D] and the number of tokens."""
    n, hq, d = q.shape
    n_blocks, bs, heads = k.shape[:3]
    g = hq // heads
    out, lse, status = np.zeros((n, hq, d)), np.full((n, hq), -np.inf), np.zeros(n, np.int64)
    slack = [[(0.0, np.zeros(d), 0)] * hq for _ in range(n)]
    for i in range(n):
        for h in range(heads):
            at, st = live_tokens(table[i], int(lens[i]), bs, n_blocks, width, None if blocks is None else blocks[i, h])
            status[i] = min(status[i], st)
            if not at:
                continue
            rows = np.array(at)
            ks, vs = k[rows[:, 0], rows[:, 1], h], v[rows[:, 0], rows[:, 1], h]
            for x in range(h * g, (h + 1) * g):
                s = scale * (ks @ q[i, x])
                top = s.max()
                w = np.exp(s - top)
                p = w / w.sum()
                out[i, x], lse[i, x] = p @ vs, top + math.log(w.sum())
                slack[i][x] = (abs(scale) * float((np.abs(ks) @ np.abs(q[i, x])).max()), p @ np.abs(vs), len(at))
    return out, lse, status, slack
