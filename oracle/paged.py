"""Paged key-value cache in numpy fp64, token by token: appending, one-token
attention, eviction by accumulated attention weight.

A cache is a dict: k, v [pages, page_size, H_kv, d], w [pages, H_kv, page_size],
table int [N, max_pages], lens int [N].  A table entry outside the pool means
that page's tokens are left out; a length outside the table's reach means an
empty sequence.
"""

from __future__ import annotations

import numpy as np


def place(c, n, j):
    """(page, slot) of token j of sequence n, or None where its page is bad."""
    P = c["k"].shape[1]
    page = int(c["table"][n, j // P])
    return (page, j % P) if 0 <= page < c["k"].shape[0] else None


def length(c, n):
    x = int(c["lens"][n])
    return x if 0 <= x <= c["table"].shape[1] * c["k"].shape[1] else 0


def append(c, k, v, cu=None):
    """In place on c (k, v, w, lens)."""
    N, cap = c["table"].shape[0], c["table"].shape[1] * c["k"].shape[1]
    cu = list(range(N + 1)) if cu is None else list(cu)
    if cu[0] != 0 or cu[-1] != k.shape[0] or any(b < a for a, b in zip(cu, cu[1:])):
        return
    for n in range(N):
        x, y = int(c["lens"][n]), cu[n + 1] - cu[n]
        if x < 0 or x + y > cap:
            continue
        for i in range(y):
            at = place(c, n, x + i)
            if at is not None:
                c["k"][at], c["v"][at] = k[cu[n] + i], v[cu[n] + i]
                c["w"][at[0], :, at[1]] = 0
        c["lens"][n] = x + y


def attention(c, q, scale, window=0, add_weights=False):
    """Returns o, lse, and what an error bound needs: a = sum_j p_j |v_j| [N, H, d] and
    smax = max_j |scale| sum_i |q_i k_ji| [N, H].  add_weights updates c["w"]."""
    N, H, d = q.shape
    G = H // c["k"].shape[2]
    o, a = np.zeros((N, H, d)), np.zeros((N, H, d))
    lse, smax = np.full((N, H), -np.inf), np.zeros((N, H))
    add = []
    for n in range(N):
        x = length(c, n)
        js = range(max(0, x - window) if window else 0, x)
        at = [p for p in (place(c, n, j) for j in js) if p is not None]
        if not at:
            continue
        pg, sl = np.array([p[0] for p in at]), np.array([p[1] for p in at])
        for h in range(H):
            k, v = c["k"][pg, sl, h // G], c["v"][pg, sl, h // G]
            s = scale * (k @ q[n, h])
            smax[n, h] = abs(scale) * np.max(np.abs(k) @ np.abs(q[n, h]))
            m = s.max()
            if np.isneginf(m):
                continue
            e = np.exp(s - m)
            lse[n, h] = m + np.log(e.sum())
            p = e / e.sum()
            o[n, h], a[n, h] = p @ v, p @ np.abs(v)
            add.append((pg, sl, h // G, p))
    if add_weights:
        for pg, sl, h, p in add:
            np.add.at(c["w"], (pg, h, sl), p)
    return o, lse, a, smax


def kept(w, length, budget, sink, recent):
    """Indices that one (sequence, head) keeps, given its weights [length]."""
    if length <= budget:
        return list(range(length))
    mid = list(range(sink, length - recent))
    key = lambda j: (np.isnan(w[j]), -w[j] if not np.isnan(w[j]) else 0.0, j)  # noqa: E731
    best = sorted(mid, key=key)[:budget - sink - recent]
    return list(range(sink)) + sorted(best) + list(range(length - recent, length))


def evict(c, budget, sink=0, recent=0, dst=None):
    """In place on c, or into dst.  Returns the kept indices [N, H_kv, budget]."""
    N, H = c["table"].shape[0], c["k"].shape[2]
    to = c if dst is None else dst
    out = np.full((N, H, budget), -1, dtype=np.int64)
    for n in range(N):
        x = length(c, n)
        bad = x != int(c["lens"][n])
        if min(x, budget) > to["table"].shape[1] * to["k"].shape[1]:
            x, bad = 0, True
        for h in range(H):
            w = np.array([c["w"][p[0], h, p[1]] if p is not None else np.nan
                          for p in (place(c, n, j) for j in range(x))])
            idx = kept(w, x, budget, sink, recent)
            out[n, h, :len(idx)] = idx
            rows = [(place(c, n, j), place(to, n, i)) for i, j in enumerate(idx)]
            held = [(b, c["k"][a[0], a[1], h].copy(), c["v"][a[0], a[1], h].copy(), c["w"][a[0], h, a[1]])
                    for a, b in rows if a is not None and b is not None]
            for b, k, v, wt in held:
                to["k"][b[0], b[1], h], to["v"][b[0], b[1], h], to["w"][b[0], h, b[1]] = k, v, wt
        if not (bad and dst is None):
            to["lens"][n] = min(x, budget)
    return out
