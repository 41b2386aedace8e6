"""Token rows to sorted rows, and the gradients of the way there and back
(oracle; test infrastructure only)."""
from __future__ import annotations

import numpy as np


def permute(x: np.ndarray, pair_to_sorted: np.ndarray, topk: int):
    """xs[pair_to_sorted[t*topk + j]] = x[t] for every pair with an expert.
    Returns (xs [T*topk][N] of x's type, zero where nothing was written,
    written bool [T*topk])."""
    p2s = np.asarray(pair_to_sorted, np.int64)
    p = np.nonzero(p2s >= 0)[0]
    xs = np.zeros((p2s.size, x.shape[1]), x.dtype)
    written = np.zeros(p2s.size, bool)
    xs[p2s[p]] = x[p // topk]
    written[p2s[p]] = True
    return xs, written


def permute_backward(dxs: np.ndarray, pair_to_sorted: np.ndarray, topk: int):
    """Each token's row of xs was copied to its pairs' rows, so its gradient
    is the sum of theirs.  Returns float64 [T][N]."""
    p2s = np.asarray(pair_to_sorted, np.int64).reshape(-1, topk)
    dxs = np.asarray(dxs, np.float64)
    dx = np.zeros((p2s.shape[0], dxs.shape[1]))
    for j in range(topk):
        v = p2s[:, j] >= 0
        dx[v] += dxs[p2s[v, j]]
    return dx


def scatter_combine_backward(dout, y, pair_to_sorted, topk_weights):
    """Gradients of combine.scatter_combine, out[t] = sum_j w[t, j] * y[s(t, j)]:
    dy[s] = w[t, j] * dout[t], dw[t, j] = dout[t] . y[s].  Returns float64
    (dy [P][N], zero rows where no pair lands, dw [T][topk], zero for pairs
    without an expert)."""
    w = np.asarray(topk_weights, np.float64)
    T, k = w.shape
    p2s = np.asarray(pair_to_sorted, np.int64)
    dout, y = np.asarray(dout, np.float64), np.asarray(y, np.float64)
    dy, dw = np.zeros_like(y), np.zeros(T * k)
    p = np.nonzero(p2s >= 0)[0]
    dy[p2s[p]] = w.reshape(-1)[p, None] * dout[p // k]
    dw[p] = (dout[p // k] * y[p2s[p]]).sum(axis=1)
    return dy, dw.reshape(T, k)
