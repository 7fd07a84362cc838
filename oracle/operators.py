"""MXFP4 and router-balance operators in float64 (NumPy), from their definitions.

MXFP4 (include/qmoe.h): blocks of 32 inputs, E2M1 codes (byte j: input 2j in the
low nibble) and one E8M0 scale byte per block, value 2^(s - 127), 255 NaN.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_VALUE = np.concatenate([E2M1, -E2M1])


def mx_quantize(x: np.ndarray):
    """x [rows][cols] -> codes uint8 [rows][16 nb], scale uint8 [rows][nb]."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    v = np.zeros((rows, nb * 32))
    v[:, :cols] = x
    v = v.reshape(rows, nb, 32)
    bad = ~np.isfinite(v).all(2)
    v = np.where(bad[:, :, None], 0.0, v)
    amax = np.abs(v).max(2)
    _, ex = np.frexp(amax)                       # amax = m 2^ex, m in [0.5, 1)
    s = np.where(amax > 0, np.clip(ex - 3, -127, 127), -127)
    a = np.abs(np.ldexp(v, -s[:, :, None]))
    dist = np.abs(a[..., None] - E2M1)           # nearest, ties to the even code
    code, best = dist.argmin(-1), dist.min(-1)
    for c in range(0, 8, 2):
        code = np.where(dist[..., c] == best, c, code)
    code = (code + 8 * np.signbit(v)).astype(np.uint8)
    code[bad] = 0
    code = code.reshape(rows, nb * 32)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(bad, 255, s + 127).astype(np.uint8)


def mx_values(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """codes [..., k/2], scale [..., k/32] -> float64 [..., k]."""
    v = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
    v[..., 0::2] = _VALUE[codes & 15]
    v[..., 1::2] = _VALUE[codes >> 4]
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def row_experts(offsets, rows: int) -> np.ndarray:
    """Expert of each row, -1 from offsets[-1] on."""
    e = np.searchsorted(np.asarray(offsets)[1:], np.arange(rows), side="right")
    return np.where(np.arange(rows) < offsets[-1], e, -1)


def grouped_matmul(a, w, offsets, index=None, rows=None, transpose=False):
    """out[r] = a[index[r]] @ w[e(r)].T (transpose: @ w[e(r)]) for the rows that
    belong to an expert (others 0), and the same sums over magnitudes, which
    bound the rounding of a sum in any order.  An index outside `a` reads zeros."""
    rows = (len(index) if index is not None else a.shape[0]) if rows is None else rows
    e = row_experts(offsets, rows)
    src = np.arange(rows) if index is None else np.asarray(index)
    ok = (src >= 0) & (src < a.shape[0])
    x = np.where(ok[:, None], a[np.where(ok, src, 0)], 0.0)
    cols = w.shape[2] if transpose else w.shape[1]
    out, mag = np.zeros((rows, cols)), np.zeros((rows, cols))
    for i in np.unique(e[e >= 0]):
        m = w[i] if transpose else w[i].T
        out[e == i] = x[e == i] @ m
        mag[e == i] = np.abs(x[e == i]) @ np.abs(m)
    return out, mag


def _log_sigmoid(x):
    return np.where(x >= 0, -np.log1p(np.exp(-np.abs(x))), x - np.log1p(np.exp(-np.abs(x))))


def shares(logits: np.ndarray, score: str) -> np.ndarray:
    a = _log_sigmoid(logits) if score == "sigmoid" else logits
    p = np.exp(a - a.max(1, keepdims=True))
    return p / p.sum(1, keepdims=True)


def balance(logits, ids, seq_offsets, coef, score, dloss=1.0):
    """(loss, counts [S][E], tokens [S], dlogits [T][E])."""
    T, E = logits.shape
    S = len(seq_offsets) - 1
    counts, tokens = np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    grad, loss = np.zeros((T, E)), 0.0
    for s in range(S):
        lo, hi = seq_offsets[s], seq_offsets[s + 1]
        pick = (ids[lo:hi] >= 0) & (ids[lo:hi] < E)
        t = lo + np.nonzero(pick.any(1))[0]
        if len(t) == 0:
            continue
        counts[s] = np.bincount(ids[lo:hi][pick], minlength=E)
        tokens[s] = len(t)
        f = E * counts[s] / counts[s].sum()
        x = logits[t]
        p = shares(x, score)
        loss += coef / S * float((p @ f).sum()) / len(t)
        d = np.exp(_log_sigmoid(-x)) if score == "sigmoid" else 1.0
        grad[t] = dloss * coef / (S * len(t)) * p * (f - (p @ f)[:, None]) * d
    return loss, counts, tokens, grad
