"""SiLU·up of f32 rows keeps f32's bits, whatever the gate, and the gated or plain
product its range, whatever the scales.

With u = 2^-24: exp(-|g|) to 1 ulp, 2 u; the sum, the reciprocal and the product
by exp, 1 u each: sig(g) and sig(-g) to 5 u (2 u of exp count by at most 1/2 in
1 / (1 + exp), 3 u there).  h = g sig u: two products more, 7 u; taken as 8.
dgu's first half, d u (s + t c) with t = g s and c = sig(-g): 5 u of s, 5 + 1 + 5 u
of t c, the sum and two products 3 u of all: at most 14 u |d u| (s + |t| c).  Its
second half d t: 7 u, taken as 8.  Numbers below 2^-126 are multiples of 2^-149:
half a step each in exp and the products that enlarge it, by at most |g| and |u|,
or what |d u| makes of it.  A gated GEMM's gate and up are three roundings off
(the sum's conversion, two products), which silu takes on by 1 + |g| c: (8 + 3 (1 +
|g| c) + 3) u |h|."""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import host
from tests.test_gpu_int8 import U, Experts, within
from tests.test_gpu_permute import F32, half_step

pytestmark = pytest.mark.gpu

mq = pytest.importorskip("quantized_moe_grouped_route_amd")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mq.lib()


def sigmoids(g):
    e = np.exp(-np.abs(g))
    big, small = 1 / (1 + e), e / (1 + e)
    return np.where(g < 0, small, big), np.where(g < 0, big, small)


def check(gu, dh, h, dgu, what):
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    s, c = sigmoids(g)
    floor = 2.0 ** -148 * (1 + np.abs(g)) * (1 + np.abs(u))
    ref = oracle.silu_gate(gu)
    within(h, ref, half_step(ref, F32) + 8 * U * np.abs(ref) + floor, (what, "h"))
    if dgu is None:
        return
    ref = oracle.silu_gate_backward(dh, gu)
    t, a = np.abs(g * s), np.abs(dh * u)
    within(dgu, ref, half_step(ref, F32) + np.concatenate([14 * U * a * (s + t * c), 8 * U * np.abs(dh) * t], 1) +
           np.concatenate([floor, floor], 1) * (1 + np.abs(np.concatenate([dh, dh], 1))), (what, "dgu"))


@pytest.mark.parametrize("P,I", [(1, 8), (37, 1000), (300, 4096)])
@pytest.mark.parametrize("span", [4.0, 30.0, 110.0])
def test_gates_of_every_size(P, I, span):
    rng = np.random.default_rng(P + I)
    gu = torch.from_numpy(np.concatenate([rng.uniform(-span, span, (P, I)), rng.standard_normal((P, I))], 1)
                          .astype(np.float32)).cuda()
    dh = torch.from_numpy(rng.standard_normal((P, I)).astype(np.float32)).cuda()
    h, ck, cs = mq.moe_silu_mul(gu, checkpoint=True)
    d, again = mq.moe_silu_mul_backward(dh, gu=gu, need_h=True)
    check(host(gu), host(dh), host(h), host(d), "columns")
    assert torch.equal(again, h)
    # the checkpoint's values are one fp32 product
    B = cs.shape[1] // 2
    col = np.arange(I) // 128
    kept = (ck.cpu().numpy().astype(np.float32) * cs.cpu().numpy()[:, np.concatenate([col, B + col])]).astype(np.float64)
    d, again = mq.moe_silu_mul_backward(dh, ck=ck, cs=cs, need_h=True)
    check(kept, host(dh), host(again), host(d), "checkpoint")
    assert torch.equal(mq.moe_silu_mul_again(ck, cs, dtype=F32), again)


@pytest.mark.parametrize("sched", ["decode", "prefill"])
def test_gated_gemm_of_large_gates(sched):
    p = Experts(51, 90, 2, 5, 544, 1152, "token", "repeat", 0.1)
    p.d["sa"] *= 40                                          # gates to about +-100
    y = oracle.grouped_gemm_qint8(p.a, host(p.d["sa"]), "token", p.w, p.sw, p.off, p.srt, p.k)["y"]
    g = y[:, :272]
    assert np.abs(g).max() > 60
    s, c = sigmoids(g)
    ref = oracle.silu_gate(y)
    h = host(p.run(F32, act="silu_mul", sched=sched))[:p.n]
    floor = 2.0 ** -148 * (1 + np.abs(g)) * (1 + np.abs(y[:, 272:]))
    within(h, ref, half_step(ref, F32) + (8 + 3 * (1 + np.abs(g) * c) + 3) * U * np.abs(ref) + floor)


@pytest.mark.parametrize("sched", ["decode", "prefill"])
@pytest.mark.parametrize("rows", [5, 70])
def test_scales_whose_product_leaves_the_range(rows, sched):
    # powers of two, so that every result within the range is exact
    N, K = 64, 128
    a = torch.full((rows, K), 64, dtype=torch.int8, device="cuda")
    a[1] = 0                                                  # a row of zeros: zeros, whatever its scale
    w = torch.full((1, N, K), 64, dtype=torch.int8, device="cuda")
    w[0, 3::4] = 0                                            # and so are columns of zeros
    acc = 64.0 * 64 * K                                       # 2^19
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    for ea, ew in ((120, 90), (127, 95), (121, -148), (-130, -20), (-149, 95), (100, -149), (-60, -80)):
        # ea, ew at the ends: a_scale * w_scale leaves the range, or keeps no bits
        sa = torch.full((rows,), 2.0 ** ea, dtype=torch.float64).float().cuda()
        sw = torch.full((1, N), 2.0 ** ew, dtype=torch.float64).float().cuda()
        exact = acc * 2.0 ** ea * 2.0 ** ew
        want = np.full((rows, N), np.float32(exact) if exact < 2.0 ** 128 else np.float32("inf"), np.float32)
        want[1], want[:, 3::4] = 0, 0
        y = mq.grouped_gemm_qint8(a, sa, w, sw, off, None, 1, out_dtype=F32, sched=sched)
        assert np.array_equal(y.cpu().numpy(), want), (ea, ew)
        # gates of zero beside any scale: zero; ups of zero too, where the gate is finite
        g = mq.grouped_gemm_qint8(a, sa, w, sw, off, None, 1, act="silu_mul", out_dtype=F32, sched=sched).cpu().numpy()
        assert not g[1].any()
        if np.isfinite(want).all():
            v = want.astype(np.float64)
            assert not g[:, 3::4].any()
            ref = oracle.silu_gate(v)
            within(g.astype(np.float64), ref, half_step(ref, F32) + 20 * U * np.abs(ref) + 2.0 ** -148 * (1 + np.abs(v[:, 32:])))
