"""The paged-cache operators in float64 numpy, one unit (a sequence's KV head) at a time.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  A cache is given as plain arrays of the
rows it holds; pages, strides and storage types are the caller's.
"""
from __future__ import annotations

import numpy as np


def norm_rope(x: np.ndarray, pos: int, w: np.ndarray | None, eps: float, base: float, rd: int) -> np.ndarray:
    """One head: x / sqrt(mean(x^2) + eps) * w (w None: x), then the half-split rotation of the
    first rd dimensions by pos * base^(-2i/rd)."""
    y = x if w is None else x / np.sqrt(np.mean(x * x) + eps) * w
    a = pos * base ** (-2.0 * np.arange(rd // 2) / rd)
    out = y.copy()
    lo, hi = y[: rd // 2], y[rd // 2: rd]
    out[: rd // 2] = lo * np.cos(a) - hi * np.sin(a)
    out[rd // 2: rd] = hi * np.cos(a) + lo * np.sin(a)
    return out


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """q [G][d] over rows k, v [n][d]: (out [G][d], lse [G], p [G][n]); no rows: zeros and -inf."""
    if len(k) == 0:
        return np.zeros((len(q), v.shape[1])), np.full(len(q), -np.inf), np.zeros((len(q), 0))
    z = scale * (q @ k.T)
    top = z.max(1, keepdims=True)
    e = np.exp(z - top)
    total = e.sum(1, keepdims=True)
    p = e / total
    return p @ v, (top + np.log(total))[:, 0], p


def kept_rows(weight: np.ndarray, position: np.ndarray, budget: int, recent: int, sink: int) -> np.ndarray:
    """Truth values of the rows that stay."""
    n = len(weight)
    if n <= budget:
        return np.ones(n, bool)
    last = int(position.max())
    safe = (position.astype(np.int64) > last - recent) | (position < sink)
    # protected rows first, then a NaN, then by weight; the lower row among equals
    grade = np.where(safe, 2, np.where(np.isnan(weight), 1, 0))
    order = sorted(range(n), key=lambda i: (-grade[i], -weight[i] if grade[i] == 0 else 0.0, i))
    kept = np.zeros(n, bool)
    kept[order[:budget]] = True
    return kept


def moves(kept: np.ndarray, budget: int) -> list[tuple[int, int]]:
    """(to, of): given-up rows below the budget and the kept rows behind it that fill them."""
    to = [i for i in range(min(budget, len(kept))) if not kept[i]]
    of = [i for i in range(budget, len(kept)) if kept[i]]
    assert len(to) == len(of)
    return list(zip(to, of))
