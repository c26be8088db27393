"""Rotation, the 4-bit cache and log probabilities written out in numpy (64 bits; the 4-bit codes in the 32 bits that define
them), pair by pair and row by row (tests only)."""
import math

import numpy as np

from paged_ref import place, seen_rows
from workloads import round_to_bf16


def freqs(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def pairs(rot, interleaved):
    return [(2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2) for i in range(rot // 2)]


def rotate(rows, H, Hkv, freq, pos, interleaved, inverse=False):
    """(rotated rows, sum of the two magnitudes that made each value); rows [B, T, heads, D], pos [B]."""
    y, mag = rows.astype(np.float64).copy(), np.abs(rows.astype(np.float64))
    B, T = rows.shape[:2]
    for i, (a, b) in enumerate(pairs(2 * len(freq), interleaved)):
        n = np.asarray(pos, np.float64)[:, None] + np.arange(T)
        c, s = np.cos(n * freq[i])[:, :, None], np.sin(n * freq[i])[:, :, None]
        if inverse:
            s = -s
        x0, x1 = rows[:, :, : H + Hkv, a].astype(np.float64), rows[:, :, : H + Hkv, b].astype(np.float64)
        y[:, :, : H + Hkv, a] = x0 * c - x1 * s
        y[:, :, : H + Hkv, b] = x1 * c + x0 * s
        mag[:, :, : H + Hkv, a] = mag[:, :, : H + Hkv, b] = np.abs(x0) + np.abs(x1)
    return y, mag


def quantise(x):
    """(codes [.., D / 2] uint8, ranges [.., 2] fp32 of bf16 values) of rows x [.., D] of bf16 values."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        low, high = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        span = (high - low).astype(np.float32)
        fine = np.isfinite(x).all(-1, keepdims=True) & np.isfinite(span)
        scale = round_to_bf16(np.where(fine, span, 0) * np.float32(1.0 / 15.0))
        scale = np.where(scale < np.float32(2.0 ** -126), np.float32(0), scale).astype(np.float32)
        inv = np.where(scale > 0, np.float32(1.0) / np.where(scale > 0, scale, 1), 0).astype(np.float32)
        n = np.minimum(np.rint((x - low).astype(np.float32) * inv), 15)
    n = np.where(fine, n, 0).astype(np.uint8)
    ranges = np.where(fine, np.concatenate([scale, low], -1), np.nan).astype(np.float32)
    return n[..., 0::2] | (n[..., 1::2] << 4), ranges


def values(codes, ranges):
    """What they stand for, in 64 bits."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (2 * codes.shape[-1],)).astype(np.float64)
    return ranges[..., 1:].astype(np.float64) + ranges[..., :1].astype(np.float64) * n


def attend4(qkv, codes, ranges, table, lens, H, window, sinks, added=0):
    """(y, lse2, bounds of y's and lse2's errors apart from y's rounding); rows of no sequence are NaN.

    The bounds. A score is scale (q . code) + low Q: the products are exact (queries enter them times a power of two,
    in fp16; what is below 2^-34 of its largest value is lost), and a chain of at most 16 sums of at most 16 sum |q| is off by
    2^-24 of that at every step, or 2^-23 where an adder cuts off: 2^-19 16 sum |q|, times the scale; the low term adds three
    roundings. So the base-2 exponents are off by d, the weights by the factor 2^(2 d), another 2^-20 for exponentials and sums.
    A weight times its scale is rounded to fp16 once, 2^-12 of it, times |code - 8| <= 8; the smallest ones to whole multiples
    of 2^-39 of 2^E, which is at most twice the largest scale or lowest value: 2^-40 8 of that for each row. The sum that
    stands for low + 8 scale takes the weights as they are. (The kernels hold such products in two parts, in a unit that follows
    the head's largest: paged4_ref.attend_rows has those closer bounds.)
    """
    pages, _, Hkv, page, half = codes.shape
    D, B, G = 2 * half, len(lens), H // Hkv
    held = values(codes, ranges)
    y, lse2 = np.full((B, H, D), np.nan), np.full((B, H), np.nan)
    ey, el = np.zeros((B, H, D)), np.zeros((B, H))
    rows = qkv.reshape(B, H + 2 * Hkv, D).astype(np.float64)
    c = 1.0 / (math.sqrt(D) * math.log(2.0))
    for b in range(B):
        if lens[b] < 0:
            continue
        seen = seen_rows(int(lens[b]) + added, window, sinks)
        if not seen:
            y[b], lse2[b] = 0.0, -np.inf
            continue
        where = [place(table[b], page, r) for r in seen]
        pg, sl = np.array([p for p, _ in where]), np.array([s for _, s in where])
        for j in range(Hkv):
            k, u = held[pg, 0, j, sl], held[pg, 1, j, sl]
            kr, ur = np.abs(ranges[pg, 0, j, sl].astype(np.float64)), np.abs(ranges[pg, 1, j, sl].astype(np.float64))
            for h in range(j * G, (j + 1) * G):
                q = rows[b, h]
                z = (k @ q) * c
                m = z.max()
                e = np.exp2(z - m)
                a = e / e.sum()
                y[b, h], lse2[b, h] = a @ u, m + math.log2(e.sum())
                qa = np.abs(q).sum()
                d = c * qa * float((2.0 ** -15 * kr[:, 0] + 2.0 ** -22 * (16 * kr[:, 0] + kr[:, 1])).max())
                el[b, h] = d + 2.0 ** -20 + 2.0 ** -22 * abs(lse2[b, h])
                off = 2 * (2 * d * math.log(2.0) + 2.0 ** -20)
                ey[b, h] = float(a @ (8 * ur[:, 0])) * 2.0 ** -12 + float(a @ (16 * ur[:, 0] + ur[:, 1])) * off + \
                    len(seen) * 2.0 ** -36 * float(ur.max()) / float(e.sum())
    return y.reshape(B, H * D), lse2, ey.reshape(B, H * D), el


def logprobs(z, targets, K=0):
    """(logp, entropy, top ids, top logp, softmax, ln softmax) of rows z, in 64 bits; rows without a finite log-sum-exp: NaN
    and ids of -1."""
    z = np.asarray(z, np.float64)
    M, V = z.shape
    logp, entropy = np.full(M, np.nan), np.full(M, np.nan)
    ids, top = np.full((M, K), -1, np.int64), np.full((M, K), np.nan)
    p, lp = np.full((M, V), np.nan), np.full((M, V), np.nan)
    for i in range(M):
        t = -1 if targets is None else int(targets[i])
        if np.isnan(z[i]).any() or z[i].max() in (np.inf, -np.inf):
            continue
        lp[i] = z[i] - z[i].max()
        lp[i] -= math.log(math.fsum(np.exp(lp[i])))
        p[i] = np.exp(lp[i])
        entropy[i] = -math.fsum(x * y for x, y in zip(p[i], lp[i]) if x > 0)
        logp[i] = lp[i, t] if 0 <= t < V else 0.0
        order = sorted(range(V), key=lambda j: (-z[i, j], j))[:K] if K else []
        ids[i], top[i] = order, lp[i, order]
    return logp, entropy, ids, top, p, lp


def logprobs_grad(p, lp, entropy, targets, dlogp, dentropy):
    """The gradient of the logits, from what logprobs gives."""
    M, V = p.shape
    g = np.zeros((M, V))
    for i in range(M):
        t = -1 if targets is None else int(targets[i])
        if dlogp is not None and 0 <= t < V:
            g[i] -= dlogp[i] * p[i]
            g[i, t] += dlogp[i]
        if dentropy is not None:
            g[i] -= dentropy[i] * np.where(p[i] > 0, p[i] * (np.where(p[i] > 0, lp[i], 0) + entropy[i]), 0.0)
        if np.isnan(entropy[i]):
            g[i] = np.nan
    return g
