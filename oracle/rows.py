"""The row operators in float64 (NumPy), from their definitions: norm with the
residual's addition, rows into expert order and back, SwiGLU, their gradients.

Each gradient comes with `mag`, the same sums over magnitudes, which bound the
rounding of a sum in any order.
"""
from __future__ import annotations

import numpy as np


def rmsnorm(h, w, eps):
    """h [rows][cols] (the residual already added) -> y, 1 / rms [rows][1]."""
    m = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return h * m * w, m


def rmsnorm_grad(dy, h, w, eps, dh=None):
    """-> dx, dw and magnitudes of both."""
    m = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    g = dy * w
    dx = m * (g - h * (m * m * (g * h).mean(1, keepdims=True)))
    mag = m * (np.abs(g) + np.abs(h) * (m * m * np.abs(g * h).mean(1, keepdims=True)))
    if dh is not None:
        dx, mag = dx + dh, mag + np.abs(dh)
    t = dy * h * m
    return dx, t.sum(0), mag, np.abs(t).sum(0)


def e4m3_grid():
    """The non-negative values of E4M3: 2^-9 steps below 2^-6, eighths above, up to 448."""
    return np.array([k * 2.0 ** -9 for k in range(8)] +
                    [(1 + k / 8) * 2.0 ** e for e in range(-6, 9) for k in range(8)][:-1])


def e4m3_rows(x):
    """x [rows][cols] -> values of the codes, scale [rows]; a row with an infinity
    or a NaN: 0 and NaN."""
    grid = e4m3_grid()
    top = np.abs(x).max(1)
    bad = ~np.isfinite(top)
    scale = np.maximum(np.where(bad, 1.0, top) / 448, 2.0 ** -126)
    v = np.where(bad[:, None], 0.0, x) / scale[:, None]
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    up = (grid[hi] - a < a - grid[lo]) | ((grid[hi] - a == a - grid[lo]) & (hi % 2 == 0))     # ties: the even code
    return np.copysign(np.where(up, grid[hi], grid[lo]), v), np.where(bad, np.nan, scale)


def dispatch(x, inv, rows):
    """`rows` with x[t] at every slot inv[t][i] that lies in it."""
    out = np.array(rows)
    for t, i in zip(*np.nonzero((inv >= 0) & (inv < len(out)))):
        out[inv[t, i]] = x[t]
    return out


def collect(rows, inv, w=None, add=None, cols=None):
    """-> y [T][cols] and the sums of magnitudes."""
    T, K = inv.shape
    y = np.zeros((T, rows.shape[1] if cols is None else cols)) if add is None else np.array(add, dtype=np.float64)
    mag = np.abs(y)
    for t, i in zip(*np.nonzero((inv >= 0) & (inv < len(rows)))):
        term = rows[inv[t, i]] * (1.0 if w is None else w[t, i])
        y[t] += term
        mag[t] += np.abs(term)
    return y, mag


def collect_grad(dy, inv, rows, w=None, drows=None):
    """-> drows (given rows where no pick falls), dw [T][K], and dw's magnitudes."""
    out = np.zeros(rows.shape) if drows is None else np.array(drows)
    dw, mag = np.zeros(inv.shape), np.zeros(inv.shape)
    for t, i in zip(*np.nonzero((inv >= 0) & (inv < len(rows)))):
        s = inv[t, i]
        dw[t, i], mag[t, i] = dy[t] @ rows[s], np.abs(dy[t]) @ np.abs(rows[s])
        out[s] = dy[t] * (1.0 if w is None else w[t, i])
    return out, dw, mag


def swiglu(gu):
    g, u = np.split(gu, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def swiglu_grad(gu, dh):
    """-> dgu and its magnitudes (the gate's slope before 1 and g (1 - s) cancel)."""
    g, u = np.split(gu, 2, axis=1)
    with np.errstate(over="ignore"):
        s, t = 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))
    dg = dh * u * s * (1 + g * t)
    mag = np.abs(dh * u * s) * (1 + np.abs(g) * t)
    return np.concatenate([dg, dh * g * s], 1), np.concatenate([mag, np.abs(dh * g * s)], 1)
