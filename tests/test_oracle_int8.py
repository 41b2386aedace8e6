"""The oracle of the 8-bit integer experts, against definitions written apart
from it: exact rational arithmetic, pair by pair sums, torch's activation and
differences."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
import synth


def _nearest_even(q: Fraction) -> int:
    f = q.numerator // q.denominator
    r = q - f
    return f + (1 if r > Fraction(1, 2) or (r == Fraction(1, 2) and f % 2) else 0)


def test_quantizer_against_exact_division():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((6, 40)) * np.exp(rng.standard_normal((6, 1)))).astype(np.float32)
    q, s = oracle.quantize_int8(x)
    for r in range(6):
        m = max(abs(Fraction(float(v))) for v in x[r])
        assert abs(Fraction(float(s[r])) - m / 127) <= m / 127 * Fraction(1, 2 ** 24)
        for v, c in zip(x[r], q[r]):
            t = Fraction(float(v)) * 127 / m
            # the two fp32 roundings move t by less than 2^-16: a code differs only where t is that near a border
            border = abs(t - (t.numerator // t.denominator) - Fraction(1, 2)) < Fraction(1, 2 ** 15)
            assert int(c) == _nearest_even(t) or border
        assert abs(q[r]).max() == 127


@pytest.mark.parametrize("row,scale", [
    ([0.0, 0.0], 1.0), ([2.0 ** -121, -2.0 ** -130], 1.0), ([2.0 ** -120, 0.0], 2.0 ** -120 / 127),
    ([3.0e38, -3.0e38], 3.0e38 / 127), ([np.inf, 1.0], np.nan), ([1.0, np.nan], np.nan), ([-np.inf, np.nan], np.nan),
])
def test_quantizer_edges(row, scale):
    q, s = oracle.quantize_int8(np.array([row], np.float32))
    assert np.array_equal(s, np.array([scale], np.float32), equal_nan=True)
    if scale == 1.0:
        assert not q.any()


@pytest.mark.parametrize("a_row", ["token", "sorted"])
def test_product_pair_by_pair(a_row):
    rng = np.random.default_rng(1)
    T, k, E, N, K = 9, 3, 4, 6, 5
    ids = np.where(rng.random((T, k)) < 0.3, -1, synth.uniform_ids_with_repeats(rng, T, k, E)).astype(np.int32)
    off, srt, p2s, _ = oracle.route_prep(ids, E)
    a = rng.integers(-128, 128, (T if a_row == "token" else T * k, K)).astype(np.int8)
    w = rng.integers(-128, 128, (E, N, K)).astype(np.int8)
    sa, sw = rng.random(a.shape[0]).astype(np.float32), rng.random((E, N)).astype(np.float32)
    r = oracle.grouped_gemm_qint8(a, sa, a_row, w, sw, off, srt, k)
    for p, e in enumerate(ids.reshape(-1)):
        if e >= 0:
            s = p2s[p]
            row = p // k if a_row == "token" else s
            acc = [sum(int(x) * int(y) for x, y in zip(a[row], w[e, n])) for n in range(N)]
            assert r["acc"][s].tolist() == acc
            assert np.allclose(r["y"][s], float(sa[row]) * sw[e].astype(np.float64) * acc, rtol=1e-14)
    assert r["acc"].shape[0] == off[-1]


def test_product_gradient_against_differences():
    # dx is the gradient of sum(dy * y) towards real-valued activations
    rng = np.random.default_rng(2)
    E, N, K, off = 3, 6, 5, np.array([0, 4, 4, 7])
    w, sw = rng.integers(-128, 128, (E, N, K)).astype(np.int8), rng.random((E, N)).astype(np.float32)
    dy, base, x = rng.standard_normal((9, N)), rng.standard_normal((9, K)), rng.standard_normal((9, K))
    r = oracle.grouped_gemm_qint8_backward(dy, w, sw, off, base)

    def loss(x_):
        v = 0.0
        for s in range(7):
            e = 0 if s < 4 else 2
            v += sum(dy[s, n] * float(sw[e, n]) * float(w[e, n].astype(float) @ x_[s]) for n in range(N))
        return v + float((base[:7] * x_[:7]).sum())
    d = rng.standard_normal(x.shape)
    assert abs((loss(x + d) - loss(x - d)) / 2 - (r["dx"] * d).sum()) < 1e-8 * np.abs(r["mag"]).sum()
    assert not r["dx"][7:].any() and np.all(np.abs(r["dx"] - np.pad(base[:7], ((0, 2), (0, 0)))) <= r["mag"] + 1e-9)


@pytest.mark.parametrize("I", [8, 128, 136, 200])
def test_checkpoint_blocks(I):
    rng = np.random.default_rng(3)
    gu = (rng.standard_normal((5, 2 * I)) * np.exp(2 * rng.standard_normal((5, 2 * I)))).astype(np.float32)
    ck, cs = oracle.checkpoint(gu)
    B = -(-I // 128)
    assert cs.shape == (5, 2 * B)
    v = oracle.checkpoint_values(ck, cs)
    for half in (0, 1):
        for b in range(B):
            c = slice(half * I + 128 * b, half * I + min(128 * b + 128, I))
            q, s = oracle.quantize_int8(gu[:, c])
            assert np.array_equal(ck[:, c], q) and np.array_equal(cs[:, half * B + b], s)
            # every value within half a step of its block's scale
            assert np.all(np.abs(v[:, c] - gu[:, c]) <= s[:, None] * (0.5 + 1e-4))


def test_activation_and_gradient_against_torch_and_differences():
    rng = np.random.default_rng(4)
    gu, dh = rng.standard_normal((7, 24)) * 4, rng.standard_normal((7, 12))
    t = torch.from_numpy(gu).requires_grad_()
    h = torch.nn.functional.silu(t[:, :12]) * t[:, 12:]
    h.backward(torch.from_numpy(dh))
    assert np.allclose(oracle.silu_gate(gu), h.detach().numpy(), rtol=1e-13, atol=0)
    g = oracle.silu_gate_backward(dh, gu)
    assert np.allclose(g, t.grad.numpy(), rtol=1e-11, atol=1e-14)
    d, eps = rng.standard_normal(gu.shape), 1e-6
    diff = (dh * (oracle.silu_gate(gu + eps * d) - oracle.silu_gate(gu - eps * d))).sum() / (2 * eps)
    assert abs(diff - (g * d).sum()) < 1e-7
    # far from zero: no overflow, the limits of sig
    far = np.array([[-800.0, 800.0, 2.0, 3.0]])
    assert np.array_equal(oracle.silu_gate_backward(np.ones((1, 2)), far), [[0.0, 3.0, 0.0, 800.0]])
