"""Sliding-window attention with sinks and its derivative in numpy float64, one head at a time (tests only)."""
import math

import numpy as np


def seen(T, window, sinks):
    t, s = np.arange(T)[:, None], np.arange(T)[None, :]
    return (s <= t) & ((t - s < window) | (s < sinks))


def forward(q, k, u, window, sinks):
    """(y, log2-sum-exp, probabilities) of one head's [T, D] queries, keys and values."""
    s = np.where(seen(q.shape[0], window, sinks), q @ k.T / math.sqrt(q.shape[1]), -np.inf)
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    l = e.sum(-1, keepdims=True)
    return (e / l) @ u, (m + np.log(l))[:, 0] / math.log(2.0), e / l


def backward(q, k, u, dy, window, sinks):
    """(dq, dk, du) of sum(dy * y) for one query head."""
    y, _, a = forward(q, k, u, window, sinks)
    ds = a * (dy @ u.T - (dy * y).sum(-1, keepdims=True)) / math.sqrt(q.shape[1])
    return ds @ k, ds.T @ q, a.T @ dy
