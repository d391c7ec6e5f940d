"""fp64 CPU oracle for the paged key/value cache and its attention.

TEST INFRASTRUCTURE ONLY (see oracle/attention.py): nothing on the product
path imports it; it shares no code with the CUDA library.

Definitions (P = page size; request b's position p is row p % P of page
table[b][p // P]; an entry outside the pool is a page that is not held):

  decode   the query row at position x of request b sees the held keys at
           positions 0 .. min(x, length - 1):
             s_j = scale q . k_j,  o = softmax(s) v,  lse = log sum exp(s)
           and o = 0, lse = -inf where it sees none
  select   s_i = max_r sum_d max(q_rd, 0) hi_id + min(q_rd, 0) lo_id,
           the first and last pages, then the highest scores
  append   rows into slots; each page's lowest and highest key values
  plan     pages from the head of a ring of free pages, to its tail
"""

from __future__ import annotations

import math

import numpy as np


def n_pages_of(length, P):
    return (max(int(length), 0) + P - 1) // P


def decode(q, k, v, table, lengths, scale, pages=None):
    """q (B, H, Tq, D); k, v (n_pages, Hkv, P, D); table (B, width); lengths
    (B); pages (B, Hkv, K) or None.  Returns (o, lse, a, r): a = sum of the
    weights times |v| (what rounding errors of the weights act on), r = the
    largest scale * sum_d |q_d k_d| of a visible key (for error bounds)."""
    q = np.asarray(q, dtype=np.float64)
    B, H, Tq, D = q.shape
    n_pool, Hkv, P, _ = k.shape
    G, width = H // Hkv, table.shape[1]
    o, a = np.zeros((B, H, Tq, D)), np.zeros((B, H, Tq, D))
    lse, reach = np.full((B, H, Tq), -np.inf), np.zeros((B, H, Tq))
    for b in range(B):
        n = n_pages_of(lengths[b], P)
        for h in range(Hkv):
            if pages is None:
                logical = list(range(min(n, width)))
            else:
                logical = [int(i) for i in pages[b, h][:min(pages.shape[2], n)]]
            where = []                       # (position, page, row) of held keys
            for i in logical:
                if not 0 <= i < width or not 0 <= table[b, i] < n_pool:
                    continue
                for row in range(P):
                    if i * P + row < lengths[b]:
                        where.append((i * P + row, int(table[b, i]), row))
            for g in range(G):
                for t in range(Tq):
                    x = int(lengths[b]) - Tq + t
                    seen = [(pg, row) for pos, pg, row in where if pos <= x]
                    if not seen:
                        continue
                    pg, row = np.array(seen).T
                    keys = k[pg, h, row].astype(np.float64)
                    vals = v[pg, h, row].astype(np.float64)
                    row_q = q[b, h * G + g, t]
                    s = scale * (keys @ row_q)
                    m = s.max()
                    e = np.exp(s - m)
                    w = e / e.sum()
                    o[b, h * G + g, t] = w @ vals
                    a[b, h * G + g, t] = w @ np.abs(vals)
                    lse[b, h * G + g, t] = m + np.log(e.sum())
                    reach[b, h * G + g, t] = scale * (np.abs(keys) @ np.abs(row_q)).max()
    return o, lse, a, reach


def select(q, bounds, table, lengths, P, K, n_first, n_last):
    """q (B, H, Tq, D); bounds (n_pages, Hkv, 2, D).  Returns int32
    (B, Hkv, K); sums are rounded once (math.fsum)."""
    q = np.asarray(q, dtype=np.float64)
    bounds = np.asarray(bounds, dtype=np.float64)
    B, H, Tq, D = q.shape
    n_pool, Hkv = bounds.shape[:2]
    G, width = H // Hkv, table.shape[1]
    out = np.full((B, Hkv, K), -1, dtype=np.int32)
    for b in range(B):
        n = min(n_pages_of(lengths[b], P), width)
        for h in range(Hkv):
            if n <= K:
                out[b, h, :n] = np.arange(n)
                continue
            score = np.full(n, -np.inf)
            for i in range(n):
                pg = int(table[b, i])
                if not 0 <= pg < n_pool:
                    continue
                lo, hi = bounds[pg, h]
                for row in q[b, h * G:(h + 1) * G].reshape(-1, D):
                    with np.errstate(invalid="ignore"):
                        terms = np.where(row < 0, 0.0, row) * hi, np.where(row > 0, 0.0, row) * lo
                    terms = np.concatenate(terms)
                    if np.isnan(terms).any() or {np.inf, -np.inf} <= set(terms):
                        s = np.inf              # a NaN counts as +inf
                    else:
                        s = math.fsum(terms)
                    score[i] = max(score[i], s)
            chosen = set(range(n_first)) | set(range(n - n_last, n))
            rest = sorted((i for i in range(n) if i not in chosen), key=lambda i: (-score[i], i))
            chosen |= set(rest[:K - len(chosen)])
            out[b, h] = sorted(chosen)
    return out


def append(k_new, v_new, slots, k, v, bounds=None):
    """k_new, v_new (n, Hkv, D); k, v (n_pages, Hkv, P, D) and bounds
    (n_pages, Hkv, 2, D).  Returns new (k, v, bounds).  Tokens are taken one
    after another; one in a page's first row starts its bounds over."""
    k, v = k.copy(), v.copy()
    bounds = None if bounds is None else bounds.copy()
    n_pool, _, P, _ = k.shape
    for i, slot in enumerate(int(x) for x in slots):
        if not 0 <= slot < n_pool * P:
            continue
        page, row = divmod(slot, P)
        k[page, :, row] = k_new[i]
        v[page, :, row] = v_new[i]
        if bounds is None:
            continue
        if row == 0:
            bounds[page, :, 0] = bounds[page, :, 1] = k_new[i]
        else:
            bounds[page, :, 0] = np.minimum(bounds[page, :, 0], k_new[i])
            bounds[page, :, 1] = np.maximum(bounds[page, :, 1], k_new[i])
    return k, v, bounds


OK, INVALID, TOO_LARGE = 0, 1, 5


def plan(asked, lengths, table, ring, state, P, n_slots):
    """One step, request by request.  Returns a dict of the new arrays."""
    table, ring = table.copy(), ring.copy()
    B, width = table.shape
    n_pool = len(ring)
    head, tail = int(state[0]), int(state[1])
    taken, freed, tokens = 0, 0, 0
    status = OK
    new_table, new_ring = table.copy(), ring.copy()
    slots, positions, cu, out = [], [], [0], []
    if head < 0 or tail < head or tail - head > n_pool:
        status = INVALID
    for b in range(B):
        length, n = int(lengths[b]), int(asked[b])
        if length < 0 or (n < 0 and length > width * P):
            status = INVALID
        elif n > 0 and length + n > width * P:
            status = status or TOO_LARGE
        if status:
            continue
        if n > 0:
            for i in range(n_pages_of(length, P), n_pages_of(length + n, P)):
                new_table[b, i] = ring[(head + taken) % n_pool]
                taken += 1
            for p in range(length, length + n):
                page = int(new_table[b, p // P])
                slots.append(page * P + p % P if 0 <= page < n_pool else -1)
                positions.append(p)
            out.append(length + n)
        elif n < 0:
            for i in range(n_pages_of(length, P)):
                if 0 <= table[b, i] < n_pool:       # a page that is held
                    new_ring[(tail + freed) % n_pool] = table[b, i]
                    freed += 1
            out.append(0)
        else:
            out.append(length)
        tokens += max(n, 0)
        cu.append(tokens)
    if not status and (taken > tail - head or tokens > n_slots):
        status = TOO_LARGE
    if not status and tail - head + freed > n_pool:
        status = INVALID
    if status:
        return dict(lengths=np.array(lengths, dtype=np.int32), state=np.array([head, tail]),
                    cu=np.zeros(B + 1, dtype=np.int32), slots=np.full(n_slots, -1),
                    positions=np.full(n_slots, -1), status=status, table=table, ring=ring)
    fill = [-1] * (n_slots - tokens)
    return dict(lengths=np.array(out, dtype=np.int32), state=np.array([head + taken, tail + freed]),
                cu=np.array(cu), slots=np.array(slots + fill), positions=np.array(positions + fill),
                status=OK, table=new_table, ring=new_ring)
