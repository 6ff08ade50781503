"""Attention mass and the eviction that goes by it (oracle; test infrastructure only).

mass[j] = decay * old[j] (0 for the step's own positions) + the sum over the
step's tokens t that see j and the query heads of the kv head of
e^(q . k_hat_j / 16 - lse).  An eviction keeps, of L positions, the last n_recent,
the first n_sink and the largest masses between them (the lowest position on equal
masses, NaN below everything), n = min(L, budget) in all; the recent positions go
first, then the sinks, where n is smaller than both.
"""
from __future__ import annotations

import numpy as np


def scores(q_rot: np.ndarray, k_hat: np.ndarray, n_ctx: int, group: int) -> np.ndarray:
    """Masked float64 scores [T * group, L] of one kv head; q_rot [T, group, D] in the cache's basis."""
    T, L = q_rot.shape[0], k_hat.shape[0]
    s = (q_rot.reshape(T * group, -1).astype(np.float64) @ np.asarray(k_hat, np.float64).T) / 16.0
    t = np.arange(T * group)[:, None] // group
    return np.where(np.arange(L)[None, :] <= n_ctx + t, s, -np.inf)


def log_sum_exp(s: np.ndarray) -> np.ndarray:
    m = s.max(axis=1)
    return m + np.log(np.exp(s - m[:, None]).sum(axis=1))


def mass(old: np.ndarray, s: np.ndarray, lse: np.ndarray, decay: float, n_ctx: int) -> np.ndarray:
    """New mass [L] of one kv head from its scores [R, L] and lse [R]."""
    new = np.exp(s - np.asarray(lse, np.float64)[:, None]).sum(axis=0)
    if decay > 0:
        new[:n_ctx] += decay * np.asarray(old, np.float64)[:n_ctx]
    return new


def keep(m: np.ndarray, budget: int, n_sink: int, n_recent: int) -> np.ndarray:
    """Ascending kept positions of a row of masses m [L]."""
    L = m.shape[0]
    n = min(L, budget)
    recent = min(n_recent, n)
    sink = min(n_sink, n - recent)
    free = np.arange(sink, L - recent)
    w = np.asarray(m, np.float64)[free]
    nan = np.isnan(w)
    order = sorted(range(len(free)), key=lambda i: (nan[i], -w[i] if not nan[i] else 0.0, i))
    chosen = free[sorted(order[: n - sink - recent])]
    return np.concatenate([np.arange(sink), chosen, np.arange(L - recent, L)]).astype(np.int64)
