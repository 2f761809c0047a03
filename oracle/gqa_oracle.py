"""Grouped-head attention and position rotation in float64, from their formulas.

TEST INFRASTRUCTURE ONLY (same rule as ``mla_oracle``).
"""

from __future__ import annotations

import numpy as np

__all__ = ["attend", "rotate"]


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """Causal grouped-head attention of a sequence's newest tokens.

    q [n, Hq, d], the newest n of L tokens; k, v [L, Hk, d]; query head h reads
    key head h // (Hq // Hk); query i sees the keys j <= L - n + i, and one that
    sees none gives zeros. Returns (out [n, Hq, d], sum_j p_j |v_j| [n, Hq, d],
    the largest sum_e |q_e k_je| scale over the visible keys [n, Hq]); the last
    two scale the error of rounded weights and of rounded score sums.
    """
    n, Hq, d = q.shape
    L, Hk, _ = k.shape
    group = Hq // Hk
    out, mean, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros((n, Hq))
    if L == 0:
        return out, mean, size
    hidden = np.arange(L)[None, :] > (L - n + np.arange(n))[:, None]
    some = ~hidden.all(axis=1)
    for h in range(Hq):
        kh, vh = k[:, h // group], v[:, h // group]
        s = np.where(hidden, -np.inf, scale * (q[:, h] @ kh.T))[some]
        p = np.exp(s - s.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        out[some, h] = p @ vh
        mean[some, h] = p @ np.abs(vh)
        size[some, h] = np.where(hidden, 0.0, scale * (np.abs(q[:, h]) @ np.abs(kh).T))[some].max(axis=1)
    return out, mean, size


def rotate(x: np.ndarray, table: np.ndarray, positions: np.ndarray, style: str):
    """x [T, H, d]: its first D elements rotated pair by pair by the angles of the
    token's table row (table [positions, D]: cos, then sin). Pairs are (i, i + D/2)
    ("half") or (2i, 2i + 1) ("interleaved"). Returns (rotated, |a cos| + |b sin|
    per element: the size of the products that a rounded sum is made of)."""
    D = table.shape[1]
    out, size = x.copy(), np.abs(x)
    for i in range(D // 2):
        a, b = (i, i + D // 2) if style == "half" else (2 * i, 2 * i + 1)
        c, s = table[positions, i][:, None], table[positions, D // 2 + i][:, None]
        xa, xb = x[:, :, a], x[:, :, b]
        out[:, :, a], out[:, :, b] = xa * c - xb * s, xb * c + xa * s
        size[:, :, a], size[:, :, b] = np.abs(xa * c) + np.abs(xb * s), np.abs(xb * c) + np.abs(xa * s)
    return out, size
