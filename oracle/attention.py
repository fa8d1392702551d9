"""Tree attention over a paged cache in float64 numpy (include/asffn.h)."""
from __future__ import annotations

import numpy as np


def positions(table_row, page: int, n: int):
    """(page, slot) of positions 0 .. n-1 of a request."""
    p = np.arange(n)
    return np.asarray(table_row)[p // page], p % page


def append(k, v, table, lens, begin, kn, vn) -> None:
    """In place, on arrays [pages, page, heads, head_dim]."""
    page = k.shape[1]
    for r, n in enumerate(lens):
        for i, t in enumerate(range(begin[r], begin[r + 1])):
            at = (table[r][(n + i) // page], (n + i) % page)
            k[at], v[at] = kn[t], vn[t]


def tree_attention(k, v, table, lens, begin, q, anc, scale: float):
    """(o, sum_p p |v|, max_p (scale sum |q k|)) per token and head; rows that see nothing: zeros."""
    T, hq, D = q.shape
    grp = hq // k.shape[2]
    o, mass, big = np.zeros((T, hq, D)), np.zeros((T, hq, D)), np.zeros((T, hq, 1))
    for r, n in enumerate(lens):
        m = begin[r + 1] - begin[r]
        pg, sl = positions(table[r], k.shape[1], n + m)
        kr, vr = k[pg, sl].astype(np.float64), v[pg, sl].astype(np.float64)
        for t in range(begin[r], begin[r + 1]):
            see = np.concatenate([np.ones(n, bool), [(int(anc[t]) >> j) & 1 for j in range(begin[r], begin[r + 1])]]).astype(bool)
            if not see.any():
                continue
            for h in range(hq):
                qq = q[t, h].astype(np.float64)
                z = scale * (kr[see, h // grp] @ qq)
                p = np.exp(z - z.max())
                p /= p.sum()
                o[t, h] = p @ vr[see, h // grp]
                mass[t, h] = p @ np.abs(vr[see, h // grp])
                big[t, h] = abs(scale) * (np.abs(kr[see, h // grp]) @ np.abs(qq)).max()
    return o, mass, big


def received(k, table, lens, begin, q, anc, scale: float, scores):
    """(scores after the call, bound of sum_rows w x the row's score error in units of 2^-23): what each key has received."""
    out, err = np.array(scores, np.float64), np.zeros(np.shape(scores))
    D, grp = q.shape[2], q.shape[1] // k.shape[2]
    for r, n in enumerate(lens):
        m = begin[r + 1] - begin[r]
        if m == 0:
            continue
        pg, sl = positions(table[r], k.shape[1], n + m)
        kr = k[pg, sl].astype(np.float64)
        out[r, :, n:n + m] = 0
        for t in range(begin[r], begin[r + 1]):
            see = np.concatenate([np.ones(n, bool), [(int(anc[t]) >> j) & 1 for j in range(begin[r], begin[r + 1])]]).astype(bool)
            if not see.any():
                continue
            for h in range(q.shape[1]):
                qq = q[t, h].astype(np.float64)
                z = scale * (kr[see, h // grp] @ qq)
                w = np.exp(z - z.max())
                w /= w.sum()
                big = abs(scale) * (np.abs(kr[see, h // grp]) @ np.abs(qq)).max()
                at = np.flatnonzero(see)
                out[r, h // grp, at] += w
                err[r, h // grp, at] += w * big
    return out, err * (D + 16)


def evict(k, v, table, lens, scores, keep: int, first: int, recent: int, table_out):
    """In place on k and v: the kept rows on table_out's pages.  (positions, scores) kept, by request and head."""
    page, kept, best = k.shape[1], [], []
    for r, n in enumerate(lens):
        kept.append([])
        best.append([])
        for h in range(k.shape[2]):
            p = list(range(n))
            if n > keep:
                value = lambda i: -np.inf if np.isnan(scores[r, h, i]) else float(scores[r, h, i])  # noqa: E731
                # NaN is below the lowest number, too
                middle = sorted(range(first, n - recent), key=lambda i: (bool(np.isnan(scores[r, h, i])), -value(i), i))
                p = p[:first] + sorted(middle[:keep - first - recent]) + p[n - recent:]
            kept[-1].append(np.array(p, int))
            best[-1].append(scores[r, h, p])
            for j, i in enumerate(p):
                to, at = (table_out[r][j // page], j % page, h), (table[r][i // page], i % page, h)
                k[to], v[to] = k[at], v[at]
    return kept, best
