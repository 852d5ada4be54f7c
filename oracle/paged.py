"""The paged serving calls in plain numpy, 64 bits: block tables and slot maps
from request lengths, the rotated paged write, and the attention of a batch
that shares a prefix.  Written from their definitions in include/hsq.h, one
request and one token at a time."""

from __future__ import annotations

import numpy as np

from .hsq_oracle import rope

MAX_LEN = 1 << 30


def page_tables(cached, fresh, free_ids, used, table, rows, page_n, n_pages, base=0):
    """-> dict(table, slots, pos, q_start, lens, used, err); err: the words' names."""
    B, width = table.shape
    table, err = table.copy(), set()
    slots, pos = np.full(rows, -1, np.int64), np.full(rows, -1, np.int32)
    q_start, lens = np.zeros(B + 1, np.int32), np.zeros(B, np.int32)
    if not 0 <= used <= len(free_ids):
        err.add("LEN")
    used = min(max(int(used), 0), len(free_ids))
    row = 0
    for b in range(B):
        c, f = int(cached[b]), int(fresh[b])
        if c < 0 or f < 0 or c > MAX_LEN or f > MAX_LEN:
            err.add("LEN")
        c = min(max(c, 0), MAX_LEN)
        f = min(max(f, 0), MAX_LEN - c)
        if f > rows - row:  # tokens without a row are not brought
            err.add("LEN")
            f = rows - row
        lens[b] = c + f
        have, need = -(-c // page_n), -(-(c + f) // page_n)
        if need > width:
            err.add("LEN")
        for col in range(min(have, width), min(need, width)):
            if used < len(free_ids):
                page = int(free_ids[used])
                used += 1
            else:
                page = -1
            if not 0 <= page < n_pages:
                page = -1
                err.add("PAGE")
            table[b, col] = page
        q_start[b] = row
        for p in range(c, c + f):
            pos[row] = base + p
            if p // page_n < width:
                page = int(table[b, p // page_n])
                if 0 <= page < n_pages:
                    slots[row] = page * page_n + p % page_n
                else:
                    err.add("PAGE")
            row += 1
    q_start[B] = row
    return dict(table=table, slots=slots, pos=pos, q_start=q_start, lens=lens, used=used, err=err)


def page_write(pages_k, pages_v, q, k, v, pos, slots, theta, max_pos):
    """pages [n, Hkv, P, 128], q [rows, Hq, 128], k, v [rows, Hkv, 128] -> (q_out, pages_k, pages_v)."""
    n_pages, _, P, _ = pages_k.shape
    pk, pv = pages_k.astype(np.float64), pages_v.astype(np.float64)
    q_out = np.zeros(q.shape)
    for i in range(len(pos)):
        if pos[i] < 0:
            continue
        p = min(int(pos[i]), max_pos - 1)
        q_out[i] = rope(q[i].astype(np.float64), np.full(q.shape[1], p), theta)
        if 0 <= slots[i] < n_pages * P:
            page, off = divmod(int(slots[i]), P)
            pk[page, :, off] = rope(k[i].astype(np.float64), np.full(k.shape[1], p), theta)
            pv[page, :, off] = v[i]
    return q_out, pk, pv


def gather(pages, ids, count, h):
    """The first `count` tokens of head h in the pages `ids`, and which of them lie in the pool."""
    n_pages, _, P, _ = pages.shape
    at = np.arange(count)
    ids = np.asarray(ids, np.int64)[at // P] if count else np.zeros(0, np.int64)
    ok = (ids >= 0) & (ids < n_pages)
    return pages[np.where(ok, ids, 0), h, at % P].astype(np.float64), ok


def shared_attn(pages_k, pages_v, q, q_start, lens, table, prefix, prefix_len):
    """-> out [rows, Hq, 128], lse [rows, Hq], spread [rows, Hq, 128] (the weighted |values|) and
    mass [rows, Hq] (the largest sum of |q_d k_d| / sqrt(128) over the tokens seen): what error bounds
    are made of.  Rows that belong to no request: NaN."""
    Hkv, P = pages_k.shape[1], pages_k.shape[2]
    rows, Hq, D = q.shape
    r = Hq // Hkv
    out, spread = np.full((rows, Hq, D), np.nan), np.full((rows, Hq, D), np.nan)
    lse, mass = np.full((rows, Hq), np.nan), np.full((rows, Hq), np.nan)
    for h in range(Hkv):
        kp, okp = gather(pages_k, prefix, prefix_len, h)
        vp, _ = gather(pages_v, prefix, prefix_len, h)
        for b in range(len(lens)):
            s, e = int(q_start[b]), int(q_start[b + 1])
            held = min(max(int(lens[b]), 0), len(table[b]) * P)  # tokens past the table are seen by no row
            ko, oko = gather(pages_k, table[b], held, h)
            vo, _ = gather(pages_v, table[b], held, h)
            for i in range(s, e):
                own = min(max(max(int(lens[b]), 0) - (e - s) + (i - s) + 1, 0), held)
                keep = np.concatenate([okp, oko[:own]])
                k = np.concatenate([kp, ko[:own]])[keep]
                v = np.concatenate([vp, vo[:own]])[keep]
                for j in range(h * r, (h + 1) * r):
                    if not len(k):
                        out[i, j], spread[i, j], lse[i, j], mass[i, j] = 0, 0, -np.inf, 0
                        continue
                    x = k @ q[i, j].astype(np.float64) / np.sqrt(D)
                    m = x.max()
                    w = np.exp(x - m)
                    lse[i, j] = m + np.log(w.sum())
                    w /= w.sum()
                    out[i, j], spread[i, j] = w @ v, w @ np.abs(v)
                    mass[i, j] = (np.abs(k) @ np.abs(q[i, j].astype(np.float64))).max() / np.sqrt(D)
    return out, lse, spread, mass
