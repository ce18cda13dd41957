"""Oracle for the paged key/value cache (float64, CPU).

Test infrastructure only (see the package docstring).

A cache is a pool of pages [n_pages][n_kv][page_size][hd]; slot n of sequence i is slot
n % page_size of page tables[i][n // page_size].  Decode attention of one query row per head over a
sequence's first ``len`` slots; eviction keeps the last ``recent`` slots and, of the others, those
with the largest accumulated weight (equal weights: the lower slot; NaN below every number).
"""

import numpy as np


def slots_of(tables, i, n, page_size, n_pages):
    """(slots, pages, slots in their pages) of sequence i's first n slots; pages outside the pool
    are left out."""
    s = np.arange(n)
    page = np.asarray(tables)[i][s // page_size] if n else s
    ok = (page >= 0) & (page < n_pages)
    return s[ok], page[ok], s[ok] % page_size


def decode(q, kp, vp, tables, lens, scale=None):
    """q (b, n_q, hd) -> (o (b, n_q, hd), lse (b, n_q), weights: per sequence (n_kv, len), the sum
    over a group's query heads)."""
    q, kp, vp = (np.asarray(a, dtype=np.float64) for a in (q, kp, vp))
    b, n_q, hd = q.shape
    n_pages, n_kv, page, _ = kp.shape
    group = n_q // n_kv
    scale = 1.0 / np.sqrt(hd) if not scale else scale
    o = np.zeros_like(q)
    lse = np.full((b, n_q), -np.inf)
    weights = []
    cap = np.asarray(tables).shape[1] * page
    for i in range(b):
        n = min(max(int(lens[i]), 0), cap)
        slots, pages, at = slots_of(tables, i, n, page, n_pages)
        w_i = np.zeros((n_kv, n))
        for j in range(n_q):
            g = j // group
            if not len(slots):
                continue
            z = scale * (kp[pages, g, at] @ q[i, j])
            m = z.max()
            e = np.exp(z - m)
            o[i, j] = (e / e.sum()) @ vp[pages, g, at]
            lse[i, j] = m + np.log(e.sum())
            w_i[g, slots] += e / e.sum()
        weights.append(w_i)
    return o, lse, weights


def keep_slots(score, n, budget, recent):
    """The slots that stay of one (sequence, KV head), ascending; score (>= n,)."""
    if n <= budget:
        return list(range(n))
    old = n - recent
    rank = [(-np.inf if np.isnan(x) else float(x), np.isnan(x)) for x in score[:old]]
    order = sorted(range(old), key=lambda s: (rank[s][1], -rank[s][0], s))
    return sorted(order[:budget - recent]) + list(range(old, n))


def evict(score, kp, vp, tables, lens, budget, recent):
    """(keep lists per sequence and head, score, kp, vp, new lens), nothing in place."""
    score, kp, vp = (np.array(a) for a in (score, kp, vp))
    page = kp.shape[2]
    keeps, new_lens = [], []
    for i, n in enumerate(int(x) for x in lens):
        keeps.append([])
        new_lens.append(min(n, budget))
        for g in range(kp.shape[1]):
            kept = keep_slots(score[i, g], n, budget, recent)
            keeps[-1].append(kept)
            if n <= budget:
                continue
            for arr in (kp, vp):
                rows = [arr[tables[i][s // page], g, s % page].copy() for s in kept]
                for j, r in enumerate(rows):
                    arr[tables[i][j // page], g, j % page] = r
            score[i, g, :budget] = score[i, g, kept]
    return keeps, score, kp, vp, new_lens
