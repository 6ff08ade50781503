"""Rotary positions with several axes (oracle; test infrastructure only).

Pair i of rotary_dim / 2 turns by position[axis_i] * f_i.  The pairs belong to
the axes in runs of sections[a], or dealt in turn (an axis that has all its pairs
is passed over); f_i = theta^(-i / half), or per axis theta^(-k / sections[a])
for the k-th pair of axis a.  Everything in float64.
"""
from __future__ import annotations

import numpy as np


def pairs(rotary_dim: int, theta: float, sections, deal_axes: bool, axis_freqs: bool):
    """(axis, frequency) of every pair."""
    half = rotary_dim // 2
    if deal_axes:
        axis, left = [], list(sections)
        while len(axis) < half:
            for a in range(len(left)):
                if left[a]:
                    left[a] -= 1
                    axis.append(a)
    else:
        axis = np.repeat(np.arange(len(sections)), sections).tolist()
    axis = np.asarray(axis[:half])
    nth = np.array([np.sum(axis[:i] == axis[i]) for i in range(half)])
    e = nth / np.asarray(sections, np.float64)[axis] if axis_freqs else np.arange(half) / half
    return axis, np.float64(theta) ** -e


def rotate(x: np.ndarray, positions: np.ndarray, rotary_dim: int, theta: float, sections, deal_axes=False,
           axis_freqs=False, adjacent=False) -> np.ndarray:
    """x [rows, heads, 256], positions [rows, axes] -> float64 rotated rows."""
    axis, f = pairs(rotary_dim, theta, sections, deal_axes, axis_freqs)
    ang = np.asarray(positions, np.float64)[:, axis] * f
    c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
    half = rotary_dim // 2
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
    out = np.array(x, np.float64)
    u, v = out[..., a].copy(), out[..., b].copy()
    out[..., a] = u * c - v * s
    out[..., b] = u * s + v * c
    return out
