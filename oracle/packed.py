"""Rotation by positions on several axes, and attention of packed prompts, in 64 bits.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Definitions (include/fp8sm.h): pair i of a head turns by column i of the table's row
pos[axes[i]][t], after the RMS norm; attention is the softmax over what a row of a
prompt sees of it, written as plain sums.

Pins (tests/test_oracle_packed.py): equal positions on all axes give the one-axis
oracle, each axis turns its own pairs only, attention equals torch's float64 softmax
and the cache oracle on exact values, and each prompt's result is its own.
"""
import numpy as np


def norm_rope_axes(x, Hq, Hk, D, pos, cos_sin, axes, wq=None, wk=None, eps=1e-6, interleaved=False):
    """x [T, >= (Hq + Hk) D], pos [n, T], axes [rot/2] -> (y float64 [T, Hq + Hk, D],
    magnitude of each output's summands).  Rows off the table on any axis: NaN."""
    T = x.shape[0]
    y = np.asarray(x, dtype=np.float64)[:, :(Hq + Hk) * D].reshape(T, Hq + Hk, D).copy()
    if wq is not None:
        y /= np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        y[:, :Hq] *= np.asarray(wq, dtype=np.float64)
        y[:, Hq:] *= np.asarray(wk, dtype=np.float64)
    mag = np.abs(y)
    half = len(axes)
    good = np.all((pos >= 0) & (pos < cos_sin.shape[0]), axis=0)
    z, zm = y.copy(), mag.copy()
    for i, a in enumerate(axes):
        p = np.where(good, pos[a], 0)
        c, s = (np.asarray(cos_sin, dtype=np.float64)[p, j][:, None] for j in (i, i + half))
        m, k = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        z[:, :, m] = y[:, :, m] * c - y[:, :, k] * s
        z[:, :, k] = y[:, :, k] * c + y[:, :, m] * s
        zm[:, :, m] = mag[:, :, m] * np.abs(c) + mag[:, :, k] * np.abs(s)
        zm[:, :, k] = mag[:, :, k] * np.abs(c) + mag[:, :, m] * np.abs(s)
    z[~good] = np.nan
    return z, zm


def attention(q, k, v, cu, scale, causal=True, window=0):
    """q [T, Hq, D], k, v [T, H, D] -> (out, lse, spread, qk): float64 [T, Hq, D],
    [T, Hq], the probability-weighted |v| of every output and the largest sum |q||k|
    of every row (for error bounds).  Rows of no prompt: NaN."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    spread, qk = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for c0, c1 in zip(cu[:-1], cu[1:]):
        n = c1 - c0
        far = np.arange(n)[:, None] - np.arange(n)
        hidden = np.zeros((n, n), dtype=bool)
        if causal:
            hidden |= far < 0
            if window:
                hidden |= far >= window
        for h in range(Hq if n > 0 else 0):
            qh, kh, vh = q[c0:c1, h], k[c0:c1, h // G], v[c0:c1, h // G]
            with np.errstate(invalid="ignore", over="ignore"):
                s = np.where(hidden, -np.inf, qh @ kh.T * scale)
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(1, keepdims=True)
                # 0 times what a row does not see is nothing, whatever that is
                seen = np.where(hidden[:, :, None], 0.0, vh[None]) if not np.isfinite(vh).all() else None
                if seen is None:
                    out[c0:c1, h] = p @ vh / l
                else:
                    out[c0:c1, h] = (p[:, :, None] * seen).sum(1) / l
                spread[c0:c1, h] = p @ np.abs(np.nan_to_num(vh, posinf=0, neginf=0)) / l
                lse[c0:c1, h] = (m + np.log(l))[:, 0]
                qk[c0:c1, h] = np.where(hidden, 0, np.abs(qh) @ np.abs(kh).T).max(1)
    return out, lse, spread, qk
