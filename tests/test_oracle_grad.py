"""Pins of the oracle's permutation, adapters and gradients: brute force in
plain Python, and gradients against central differences of the forward
definitions (exact up to rounding: every function is a polynomial of degree
at most two in each single argument's direction, so a central difference has
no truncation error)."""
import numpy as np
import pytest

import oracle
import synth


def _tables(seed, T, k, E, skip=0.25):
    rng = np.random.default_rng(seed)
    ids = synth.uniform_ids_with_repeats(rng, T, k, E)
    ids = np.where(rng.random((T, k)) < skip, -1, ids).astype(np.int32)
    return rng, ids, oracle.route_prep(ids, E)


def _difference(f, v, direction, eps=1e-3):
    return (f(v + eps * direction) - f(v - eps * direction)) / (2 * eps)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (7, 3, 4), (12, 2, 9)])
def test_permute_and_combine_gradients(T, k, E):
    rng, ids, (off, srt, p2s, _) = _tables(T, T, k, E)
    N, P, n = 6, T * k, int(off[-1])
    x = rng.standard_normal((T, N))
    xs, written = oracle.permute(x, p2s, k)
    for s in range(P):
        assert written[s] == (s < n)
        if s < n:
            assert np.array_equal(xs[s], x[srt[s] // k])
    g, dirx = rng.standard_normal((P, N)), rng.standard_normal((T, N))
    num = _difference(lambda v: float((g * oracle.permute(v, p2s, k)[0]).sum()), x, dirx)
    assert abs(num - (oracle.permute_backward(g, p2s, k) * dirx).sum()) < 1e-9

    y, w = rng.standard_normal((P, N)), rng.standard_normal((T, k))
    dout = rng.standard_normal((T, N))
    dy, dw = oracle.scatter_combine_backward(dout, y, p2s, w)
    diry, dirw = rng.standard_normal((P, N)), rng.standard_normal((T, k))
    num = _difference(lambda v: float((dout * oracle.scatter_combine(v, p2s, w)).sum()), y, diry)
    assert abs(num - (dy * diry).sum()) < 1e-9
    num = _difference(lambda v: float((dout * oracle.scatter_combine(y, p2s, v)).sum()), w, dirw)
    assert abs(num - (dw * dirw).sum()) < 1e-9
    assert np.all(dw.reshape(-1)[p2s < 0] == 0) and np.all(dy[n:] == 0)


@pytest.mark.parametrize("a_row,out_row", [("token", "sorted"), ("sorted", "sorted"), ("token", "pair")])
def test_lora_by_rows_and_gradients(a_row, out_row):
    T, k, E, N, K, R = 9, 2, 4, 5, 7, 3
    rng, ids, (off, srt, p2s, _) = _tables(11, T, k, E)
    P, n = T * k, int(off[-1])
    x = rng.standard_normal((T if a_row == "token" else P, K))
    a, b = rng.standard_normal((E, R, K)), rng.standard_normal((E, N, R))
    base, scale = rng.standard_normal((P, N)), rng.uniform(0.5, 2, E)
    kw = dict(scale=scale, a_row=a_row, out_row=out_row)
    f = oracle.grouped_lora(x, a, b, off, srt, k, base=base, **kw)
    # pair by pair, straight from the ids
    for p, e in enumerate(ids.reshape(-1)):
        o = p if out_row == "pair" else p2s[p]
        if e < 0:
            if out_row == "pair":
                assert np.array_equal(f["out"][p], base[p]) and not f["written"][p]
            continue
        row = x[p // k] if a_row == "token" else x[p2s[p]]
        assert np.allclose(f["out"][o], base[o] + scale[e] * (b[e] @ (a[e] @ row)), atol=1e-12)
        assert np.all(np.abs(f["out"][o]) <= f["mag"][o] + 1e-12)
    assert f["written"].sum() == n

    dy = rng.standard_normal((P, N))
    g = oracle.grouped_lora_backward(dy, x, a, b, f["h"], off, srt, k, **kw)
    mask = f["written"][:, None]
    loss = lambda x_, a_, b_: float((np.where(mask, dy, 0) *
                                     oracle.grouped_lora(x_, a_, b_, off, srt, k, base=base, **kw)["out"]).sum())
    for name, v, f1 in (("da", a, lambda v: loss(x, v, b)), ("db", b, lambda v: loss(x, a, v))):
        d = rng.standard_normal(v.shape)
        assert abs(_difference(f1, v, d) - (g[name] * d).sum()) < 1e-8
    d = rng.standard_normal(x.shape)
    dx = oracle.permute_backward(g["dx"], p2s, k) if a_row == "token" else g["dx"]
    assert abs(_difference(lambda v: loss(v, a, b), x, d) - (dx * d).sum()) < 1e-8
