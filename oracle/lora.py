"""Low-rank adapters beside a projection, one per group of rows, and their
gradients (oracle; test infrastructure only).  Tables as route.route_prep
makes them: group e owns the sorted rows offsets[e] .. offsets[e+1]."""
from __future__ import annotations

import numpy as np


def _rows(offsets, sorted_pair_ids, topk, a_row, out_row):
    """(row of x, row of out) of every sorted row."""
    n = int(offsets[-1])
    s = np.arange(n)
    pair = np.asarray(sorted_pair_ids[:n], np.int64) if sorted_pair_ids is not None else s
    return (pair // topk if a_row == "token" else s), (pair if out_row == "pair" else s)


def grouped_lora(x, a, b, offsets, sorted_pair_ids, topk, *, base=None, scale=None, a_row="token", out_row="sorted",
                 P=None):
    """out[o] = base[o] + scale[e] * (x[row] . a[e]^T) . b[e]^T.

    Returns dict(h float64 [P][R], out float64 [P][N], mag [P][N]: the sum of
    the magnitudes of out's products, written bool [P]).  Rows of out without
    a group hold base (zero without one)."""
    x, a, b = (np.asarray(v, np.float64) for v in (x, a, b))
    P = len(sorted_pair_ids) if P is None else P
    E, N, R = b.shape
    rx, ro = _rows(offsets, sorted_pair_ids, topk, a_row, out_row)
    out = np.zeros((P, N)) if base is None else np.asarray(base, np.float64).copy()
    mag, h, written = np.abs(out), np.zeros((P, R)), np.zeros(P, bool)
    for e in range(E):
        i = np.arange(offsets[e], offsets[e + 1])
        sc = 1.0 if scale is None else float(scale[e])
        h[i] = x[rx[i]] @ a[e].T
        out[ro[i]] += sc * (h[i] @ b[e].T)
        mag[ro[i]] += abs(sc) * ((np.abs(x[rx[i]]) @ np.abs(a[e]).T) @ np.abs(b[e]).T)
        written[ro[i]] = True
    return dict(h=h, out=out, mag=mag, written=written)


def grouped_lora_backward(dy, x, a, b, h, offsets, sorted_pair_ids, topk, *, scale=None, a_row="token",
                          out_row="sorted"):
    """Gradients of sum(dy * out) with respect to x's row of every sorted row,
    a and b, with h as given.  Returns dict(dx [P][K], da, db and the sums of
    their products' magnitudes mdx, mda, mdb), float64."""
    dy, x, a, b, h = (np.asarray(v, np.float64) for v in (dy, x, a, b, h))
    E, R, K = a.shape
    rx, ro = _rows(offsets, sorted_pair_ids, topk, a_row, out_row)
    g = {n: np.zeros(s) for n, s in (("dx", (dy.shape[0], K)), ("da", a.shape), ("db", b.shape))}
    g.update({"m" + n: np.zeros_like(v) for n, v in list(g.items())})
    for e in range(E):
        i = np.arange(offsets[e], offsets[e + 1])
        sc = 1.0 if scale is None else float(scale[e])
        d = sc * dy[ro[i]]
        dh, mdh = d @ b[e], np.abs(d) @ np.abs(b[e])
        xi = x[rx[i]]
        g["dx"][i], g["mdx"][i] = dh @ a[e], mdh @ np.abs(a[e])
        g["da"][e], g["mda"][e] = dh.T @ xi, mdh.T @ np.abs(xi)
        g["db"][e], g["mdb"][e] = d.T @ h[i], np.abs(d).T @ np.abs(h[i])
    return g
