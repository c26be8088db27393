"""The paged cache operators written out in numpy float64, sequence by sequence and head by head (tests only)."""
import math

import numpy as np


def seen_rows(n, window, sinks):
    """The rows 0..n-1 that the newest query (row n - 1) sees."""
    return [r for r in range(n) if window == 0 or n - 1 - r < window or r < sinks]


def attend(q, k, u):
    """(y, log2-sum-exp, probabilities) of one query over the rows k, u."""
    s = (k @ q) / math.sqrt(q.shape[0])
    m = s.max()
    e = np.exp(s - m)
    return (e / e.sum()) @ u, (m + math.log(e.sum())) / math.log(2.0), e / e.sum()


def place(table_b, page, r):
    return int(table_b[r // page]), r % page


def decode(qkv, pool, weight, table, lens, H, window, sinks):
    """y, lse2 and the expected pool and weight after one step; rows of lens < 0 are NaN in y and lse2."""
    pages, _, Hkv, page, D = pool.shape
    B, G = len(lens), H // Hkv
    pool = pool.copy()
    weight = None if weight is None else weight.copy()
    y = np.full((B, H * D), np.nan)
    lse2 = np.full((B, H), np.nan)
    rows = qkv.reshape(B, H + 2 * Hkv, D)
    for b in range(B):
        if lens[b] < 0:
            continue
        pg, sl = place(table[b], page, int(lens[b]))
        pool[pg, 0, :, sl] = rows[b, H:H + Hkv]
        pool[pg, 1, :, sl] = rows[b, H + Hkv:]
        if weight is not None:
            weight[pg, :, sl] = 0.0
    for b in range(B):
        if lens[b] < 0:
            continue
        seen = seen_rows(int(lens[b]) + 1, window, sinks)
        where = [place(table[b], page, r) for r in seen]
        for j in range(Hkv):
            k = np.stack([pool[p, 0, j, s] for p, s in where])
            u = np.stack([pool[p, 1, j, s] for p, s in where])
            total = np.zeros(len(seen))
            for h in range(j * G, (j + 1) * G):
                y[b, h * D:(h + 1) * D], lse2[b, h], a = attend(rows[b, h], k, u)
                total += a
            if weight is not None:
                for (p, s), a in zip(where, total):
                    weight[p, j, s] += a
    return y, lse2, pool, weight


def evict(pool, weight, table, lens, dst_table, budget, sinks, recent):
    """(pool, weight, new_lens, kept) after an eviction."""
    pages, _, Hkv, page, D = pool.shape
    src_pool, src_weight = pool.copy(), weight.copy()
    pool, weight = pool.copy(), weight.copy()
    new_lens = np.minimum(lens, budget)
    kept = np.full((len(lens), Hkv, budget), -1, np.int64)
    for b, n in enumerate(lens):
        for j in range(Hkv):
            if n <= budget:
                rows = list(range(max(n, 0)))
            else:
                w = []
                for r in range(sinks, n - recent):
                    p, s = place(table[b], page, r)
                    v = src_weight[p, j, s]
                    w.append((bool(np.isnan(v)), 0.0 if np.isnan(v) else -v, r))    # NaN below -inf, ties by row
                w.sort()
                rows = sorted(list(range(sinks)) + list(range(n - recent, n)) +
                              [r for _, _, r in w[:budget - sinks - recent]])
            for i, r in enumerate(rows):
                p, s = place(table[b], page, r)
                q, d = place(dst_table[b], page, i)
                pool[q, :, j, d] = src_pool[p, :, j, s]
                weight[q, j, d] = src_weight[p, j, s]
                kept[b, j, i] = r
    return pool, weight, new_lens, kept
