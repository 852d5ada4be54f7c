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


# -- long contexts: rotations, summaries, selected pages -------------------------------------


def rope_frequencies(dims, theta, scaling="none", factor=1.0, original=0.0, beta_fast=32.0, beta_slow=1.0):
    """(omega [dims / 2], amplitude), one frequency at a time."""
    omega, amp = [], 1.0
    if scaling == "yarn_index":
        # the (real) index whose frequency theta^(-2 i / dims) makes t turns over the original context
        first, last = (dims / 2 * (np.log(original / (2 * np.pi)) - np.log(t)) / np.log(theta) for t in (beta_fast, beta_slow))
        first, last = (int(np.clip(x, 0, dims - 1)) for x in (np.floor(first), np.ceil(last)))
    for i in range(dims // 2):
        base = theta * factor ** (dims / (dims - 2)) if scaling == "base" else theta
        w = base ** (-2 * i / dims)
        if scaling == "linear":
            w /= factor
        elif scaling == "yarn":
            wavelength = 2 * np.pi / w
            turns = original / wavelength
            if turns <= beta_slow:
                w = w / factor
            elif turns < beta_fast:
                g = (turns - beta_slow) / (beta_fast - beta_slow)
                w = (1 - g) * w / factor + g * w
        elif scaling == "yarn_index":
            if i >= last and (last > first or i > first):
                w = w / factor
            elif i > first:
                g = (i - first) / (last - first)
                w = g * w / factor + (1 - g) * w
        omega.append(w)
    if scaling in ("yarn", "yarn_index"):
        amp = 0.1 * np.log(factor) + 1
    return np.array(omega), amp


def rotate(x, p, omega, amp, interleaved):
    """x [..., 128] at position p: the first 2 len(omega) dims as complex numbers."""
    R = 2 * len(omega)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    z = (x[..., a] + 1j * x[..., b]) * (amp * np.exp(1j * p * omega))
    y = np.array(x, np.float64)
    y[..., a], y[..., b] = z.real, z.imag
    return y


def page_write_rope(pages_k, pages_v, q, k, v, pos, slots, omega, amp, interleaved, max_pos):
    n_pages, _, P, _ = pages_k.shape
    pk, pv = pages_k.astype(np.float64), pages_v.astype(np.float64)
    q_out = np.zeros(q.shape)
    for i in range(len(pos)):
        if pos[i] < 0:
            continue
        p = min(int(pos[i]), max_pos - 1)
        q_out[i] = rotate(q[i].astype(np.float64), p, omega, amp, interleaved)
        if 0 <= slots[i] < n_pages * P:
            page, off = divmod(int(slots[i]), P)
            pk[page, :, off] = rotate(k[i].astype(np.float64), p, omega, amp, interleaved)
            pv[page, :, off] = v[i]
    return q_out, pk, pv


def summary(keys):
    """keys [n, 128] -> (codes int [128], scale)."""
    with np.errstate(invalid="ignore", over="ignore"):
        total = np.zeros(128)
        for x in keys:
            total = total + x.astype(np.float64)
        top = np.abs(total).max()
    if not top <= 2.0 ** 126:
        return np.zeros(128, int), np.inf
    if top < 2.0 ** -64:
        return np.zeros(128, int), 0.0
    return np.rint(127 * total / top).astype(int), top / (127 * len(keys))


def page_summaries(pages_k, slots, codes, scale):
    """-> codes [n_pages, Hkv, 128], scale [n_pages, Hkv] with the named pages' made anew, err."""
    n_pages, Hkv, P, _ = pages_k.shape
    codes, scale, err = codes.copy(), scale.astype(np.float64), set()
    for i, s in enumerate(slots):
        if s >= n_pages * P:
            err.add("PAGE")
        if s < 0 or s >= n_pages * P:
            continue
        nxt = slots[i + 1] if i + 1 < len(slots) else -1
        if nxt >= 0 and nxt // P == s // P:
            continue
        for h in range(Hkv):
            codes[s // P, h], scale[s // P, h] = summary(pages_k[s // P, h, : s % P + 1])
    return codes, scale, err


def row_pages(i, q_start, lens, table, page_n, prefix_len):
    """(request, own tokens that row i sees, logical pages that it sees), None for a row of no request."""
    for b in range(len(lens)):
        s, e = int(q_start[b]), int(q_start[b + 1])
        if s <= i < e:
            seen = min(max(max(int(lens[b]), 0) - (e - s) + (i - s) + 1, 0), max(int(lens[b]), 0), len(table[b]) * page_n)
            return b, seen, -(-prefix_len // page_n) + -(-seen // page_n)
    return None


def query_codes(q):
    """q [r, 128] (float32) -> whole numbers: the codes of the sum of the rows, every step as in float32."""
    x = q[0].astype(np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        for y in q[1:]:
            x = x + y.astype(np.float32)
        top = np.abs(x).max()
        if not np.isfinite(top) or top < np.float32(2.0 ** -64):
            return np.zeros(128, np.int64)
        return np.rint(x * (np.float32(127) / top)).astype(np.int64)


def page_select(codes, scale, q, q_start, lens, table, prefix, prefix_len, page_n, top, first, recent):
    """-> sel [rows, Hkv, top] (-2 in the rows of no request), err"""
    n_pages, Hkv = scale.shape
    rows, Hq, _ = q.shape
    r, err = Hq // Hkv, set()
    sel = np.full((rows, Hkv, top), -2, np.int64)
    for i in range(rows):
        at = row_pages(i, q_start, lens, table, page_n, prefix_len)
        if at is None:
            continue
        b, _, c = at
        np_ = -(-prefix_len // page_n)
        ids = np.concatenate([np.asarray(prefix, np.int64)[:np_], table[b].astype(np.int64)])[:c]
        for h in range(Hkv):
            if c <= top:
                take = list(range(c))
            else:
                cq = query_codes(q[i, h * r: (h + 1) * r])
                ranked = []
                for p in range(first, c - recent):
                    if first + recent == top:
                        break
                    if not 0 <= ids[p] < n_pages:
                        err.add("PAGE")
                        continue
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = np.float32(int(cq @ codes[ids[p], h].astype(np.int64))) * np.float32(scale[ids[p], h])
                    ranked.append((-np.inf if np.isnan(s) else -float(s), not np.isnan(s), p))
                ranked.sort()
                take = sorted(list(range(first)) + [p for _, _, p in ranked[: top - first - recent]] +
                              list(range(c - recent, c)))
            sel[i, h] = take + [-1] * (top - len(take))
    return sel, err


def page_attn(pages_k, pages_v, q, q_start, lens, table, prefix, prefix_len, sel):
    """-> out, lse, spread, mass as shared_attn's, err; rows of no request: NaN"""
    n_pages, Hkv, P, _ = pages_k.shape
    rows, Hq, D = q.shape
    r, np_, err = Hq // Hkv, -(-prefix_len // P), set()
    out, spread = np.full((rows, Hq, D), np.nan), np.full((rows, Hq, D), np.nan)
    lse, mass = np.full((rows, Hq), np.nan), np.full((rows, Hq), np.nan)
    for i in range(rows):
        at = row_pages(i, q_start, lens, table, P, prefix_len)
        if at is None:
            continue
        b, seen, c = at
        for h in range(Hkv):
            ks, vs, before = [np.zeros((0, D))], [np.zeros((0, D))], -1
            for e in sel[i, h].tolist():
                if e >= 0:
                    if e >= c or e <= before:
                        err.add("SEL")
                    else:
                        page = int(prefix[e]) if e < np_ else int(table[b][e - np_])
                        n = min(P, prefix_len - e * P if e < np_ else seen - (e - np_) * P)
                        if 0 <= page < n_pages:
                            ks.append(pages_k[page, h, :n].astype(np.float64))
                            vs.append(pages_v[page, h, :n].astype(np.float64))
                        else:
                            err.add("PAGE")
                    before = max(before, e)
            k, v = np.concatenate(ks), np.concatenate(vs)
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
    return out, lse, spread, mass, err
