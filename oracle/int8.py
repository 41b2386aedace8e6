"""Experts kept in 8-bit integers: the activation quantizer, the W8A8 grouped
product and its gradient towards the activations, and the gated activation
with its 8-bit checkpoint and gradient (oracle; test infrastructure only).
Tables as route.route_prep makes them: expert e owns the sorted rows
offsets[e] .. offsets[e+1]."""
from __future__ import annotations

import numpy as np

BLOCK = 128
TINY = np.float32(2.0 ** -120)


def quantize_int8(x):
    """Codes of the rows of x [rows][K]: amax = max |x|, scale = amax / 127,
    code = clamp(rne(x * (127 / amax)), -127, 127), each step one fp32
    operation; amax < 2^-120: zeros, scale 1; an infinity or NaN in a row:
    scale NaN (its codes are unspecified, here 0).  Returns (int8 [rows][K],
    float32 [rows])."""
    x = np.asarray(x, np.float32)
    amax = np.max(np.abs(x), axis=1) if x.shape[1] else np.zeros(x.shape[0], np.float32)
    bad = ~np.isfinite(amax)
    tiny = ~bad & (amax < TINY)
    safe = np.where(tiny | bad, np.float32(1), amax).astype(np.float32)
    recip = np.where(tiny | bad, np.float32(0), np.float32(127) / safe).astype(np.float32)
    scale = np.where(tiny, np.float32(1), safe / np.float32(127)).astype(np.float32)
    t = (np.where(bad[:, None], np.float32(0), x) * recip[:, None]).astype(np.float32)
    q = np.clip(np.rint(t), -127, 127).astype(np.int8)
    return q, np.where(bad, np.float32(np.nan), scale).astype(np.float32)


def _rows(offsets, sorted_pair_ids, topk, a_row):
    n = int(offsets[-1])
    s = np.arange(n)
    if a_row == "token" and sorted_pair_ids is not None:
        return np.asarray(sorted_pair_ids[:n], np.int64) // topk
    return s


def grouped_gemm_qint8(a, a_scale, a_row, w, w_scale, offsets, sorted_pair_ids, topk):
    """acc[s, n] = sum_k a[row(s), k] w[e, n, k]; y = a_scale * w_scale * acc.
    Returns dict(acc int64 [n][N], y float64 [n][N])."""
    row = _rows(offsets, sorted_pair_ids, topk, a_row)
    E, N, _ = w.shape
    acc, sw = np.zeros((row.size, N)), np.zeros((row.size, N))
    for e in range(E):
        i = slice(int(offsets[e]), int(offsets[e + 1]))
        acc[i] = np.asarray(a, np.float64)[row[i]] @ np.asarray(w[e], np.float64).T
        sw[i] = w_scale[e]
    return dict(acc=acc.astype(np.int64), y=np.asarray(a_scale, np.float64)[row][:, None] * sw * acc)


def grouped_gemm_qint8_backward(dy, w, w_scale, offsets, base=None):
    """dx[s] = base[s] + sum_n dy[s, n] w_scale[e, n] w[e, n], rows of no expert
    zero.  Returns dict(dx, mag: the sum of the products' magnitudes, top: the
    largest |dy * w_scale| of each row, wsum: sum_n |w[e, n]|), float64."""
    dy = np.asarray(dy, np.float64)
    P, (E, N, K) = dy.shape[0], w.shape
    r = dict(dx=np.zeros((P, K)), mag=np.zeros((P, K)), top=np.zeros(P), wsum=np.zeros((P, K)))
    for e in range(E):
        i = slice(int(offsets[e]), int(offsets[e + 1]))
        d, we = dy[i] * np.asarray(w_scale[e], np.float64), np.asarray(w[e], np.float64)
        r["dx"][i], r["mag"][i] = d @ we, np.abs(d) @ np.abs(we)
        r["top"][i] = np.abs(d).max(axis=1) if d.size else 0
        r["wsum"][i] = np.abs(we).sum(axis=0)
        if base is not None:
            r["dx"][i] += np.asarray(base, np.float64)[i]
    return r


def checkpoint(gu):
    """8-bit codes of gu [rows][2I], a scale for every 128 columns of a row's
    gate and up (quantize_int8's rule within each).  Returns (int8 [rows][2I],
    float32 [rows][2 ceil(I / 128)])."""
    gu = np.asarray(gu, np.float32)
    rows, I = gu.shape[0], gu.shape[1] // 2
    q, s = np.zeros(gu.shape, np.int8), []
    for half in (0, 1):
        for lo in range(0, I, BLOCK):
            c = slice(half * I + lo, half * I + min(lo + BLOCK, I))
            q[:, c], scale = quantize_int8(gu[:, c])
            s.append(scale)
    return q, np.stack(s, axis=1) if s else np.zeros((rows, 0), np.float32)


def checkpoint_values(ck, cs):
    """The values that a checkpoint stands for, float64 [rows][2I]."""
    I, B = ck.shape[1] // 2, cs.shape[1] // 2
    col = np.arange(I) // BLOCK
    return np.asarray(ck, np.float64) * np.asarray(cs, np.float64)[:, np.concatenate([col, B + col])]


def _sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1 / (1 + e), e / (1 + e))


def silu_gate(gu):
    """h = g sig(g) u of rows [g | u], float64."""
    I = gu.shape[1] // 2
    g, u = np.asarray(gu[:, :I], np.float64), np.asarray(gu[:, I:], np.float64)
    return g * _sigmoid(g) * u


def silu_gate_backward(dh, gu):
    """Gradient of sum(dh * silu_gate(gu)), float64 [rows][2I]."""
    I = gu.shape[1] // 2
    g, u, dh = (np.asarray(v, np.float64) for v in (gu[:, :I], gu[:, I:], dh))
    s, c = _sigmoid(g), _sigmoid(-g)
    return np.concatenate([dh * u * s * (1 + g * c), dh * g * s], axis=1)
