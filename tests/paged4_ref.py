"""Attention over given rows of a 4-bit cache in 64 bits, with the bounds of the kernels' arithmetic (tests only)."""
import math

import numpy as np

from paged_ref import place
from serving_ref import values


def attend_rows(qkv, codes, ranges, table, seen, H, product_bits=20, rounded=None):
    """(y, lse2, bounds of y's and lse2's errors apart from y's rounding); seen[b]: the rows that sequence b's query sees (None:
    no sequence, NaN).

    The bounds of scores, exponentials and sums are serving_ref.attend4's. A weight times its scale enters the product with the
    codes in two fp16 parts, both cut off: 2^-10 of 2^-10 of it is lost, times |code - 8| <= 8. The smallest ones are whole
    multiples of 2^-24, in either part, of 2^(E - 15), where 2^E is at most 2^9 times the head's largest product of a weight and
    its row's scale, or the |lowest + 8 scale| of the row: 2 2^-24 2^-15 2^9 8 = 2^-26 of that product for each row.

    product_bits: 2^-product_bits of a product may be lost. rounded(x): what stands for a weight times its scale (the weight
    against a largest one of 1), for a calculation that loses more."""
    pages, _, Hkv, page, half = codes.shape
    D, B, G = 2 * half, len(seen), H // Hkv
    held = values(codes, ranges)
    y, lse2 = np.full((B, H, D), np.nan), np.full((B, H), np.nan)
    ey, el = np.zeros((B, H, D)), np.zeros((B, H))
    rows = qkv.reshape(B, H + 2 * Hkv, D).astype(np.float64)
    c = 1.0 / (math.sqrt(D) * math.log(2.0))
    for b in range(B):
        if seen[b] is None:
            continue
        if not len(seen[b]):
            y[b], lse2[b] = 0.0, -np.inf
            continue
        where = [place(table[b], page, r) for r in seen[b]]
        pg, sl = np.array([p for p, _ in where]), np.array([s for _, s in where])
        for j in range(Hkv):
            k, u = held[pg, 0, j, sl], held[pg, 1, j, sl]
            kr, ur = (ranges[pg, w, j, sl].astype(np.float64) for w in (0, 1))
            size = np.abs(ur[:, 1]) + 8 * ur[:, 0]
            for h in range(j * G, (j + 1) * G):
                q = rows[b, h]
                z = (k @ q) * c
                m = z.max()
                e = np.exp2(z - m)
                a = e / e.sum()
                if rounded is None:
                    y[b, h] = a @ u
                else:
                    n = np.where(ur[:, :1] > 0, (u - ur[:, 1:]) / np.where(ur[:, :1] > 0, ur[:, :1], 1), 0) - 8
                    y[b, h] = (rounded(e * ur[:, 0]) @ n + e @ (ur[:, 1] + 8 * ur[:, 0])) / e.sum()
                lse2[b, h] = m + math.log2(e.sum())
                qa = np.abs(q).sum()
                d = c * qa * float((2.0 ** -15 * kr[:, 0] + 2.0 ** -22 * (16 * kr[:, 0] + np.abs(kr[:, 1]))).max())
                el[b, h] = d + 2.0 ** -20 + 2.0 ** -22 * abs(lse2[b, h])
                off = 2 * (2 * d * math.log(2.0) + 2.0 ** -20)
                ey[b, h] = float(a @ (8 * ur[:, 0])) * 2.0 ** -product_bits + \
                    float(a @ (16 * ur[:, 0] + np.abs(ur[:, 1]))) * off + len(seen[b]) * 2.0 ** -26 * float((a * size).max())
    return y.reshape(B, H * D), lse2, ey.reshape(B, H * D), el


def outside(got, y, ey):
    """Where got, rounded to bf16, is further from y than the bound and its rounding."""
    return np.abs(got - y) > 2.0 ** -8 * np.abs(y) + 1.01 * ey
