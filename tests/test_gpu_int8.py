"""The INT8 calls against the float64 oracle, at the sizes, tables and values
where they can go wrong.

Codes, scales and accumulators are exact.  Tolerances of the others, per
element, with u = 2^-24 (one fp32 rounding) and the output's own rounding half
a step:
  y = a_scale * w_scale * acc   three roundings (acc to fp32, two products): 4 u |y|
  sig = rcp(1 + exp(-g))        exp(-g) is 2^(-g log2 e) of a rounded argument (|g| log2 e u
      of the exponent, ln 2 times that of the value, and 2 u of the instruction), which
      reaches sig by the factor 1 - sig; the sum and the reciprocal 1 + 2 u:
      (8 + 2 |g|) u relative
  h = silu(g) u                 with g and u themselves 4 u off where a GEMM made them; silu's
      relative derivative is at most 1 + |g|: (16 + 8 |g|) u |h|
  gradient of silu              dh u (s + t (1 - s)), t = g s: 1 - s is off by u and by s's error:
      (16 + 4 |g|) u |dh u| (s + |t| (1 - s)) + 4 u |dh u t|; du as h
  values below 2^-118 of the other factor may be flushed (exp past 2^126): floor
  dx = base + sum d w           d as multiples of step = max|d| / 32512: half a step and, as the
      code is made with two roundings of up to 32512 units, 0.004 more: 0.51 step sum|w|; the
      roundings of d, step, the two sums' conversion and the join: 8 u mag"""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import dev, host
from tests.test_gpu_permute import BF16, F16, F32, half_step, tables, values

pytestmark = pytest.mark.gpu

mq = pytest.importorskip("quantized_moe_grouped_route_amd")

U = 2.0 ** -24


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mq.lib()


def within(got, ref, tol, what=""):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.nanmax(np.abs(got - ref) / tol)))


# ---------------------------------------------------------------- quantizer
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,K", [(0, 64), (1, 16), (3, 48), (8, 7168), (2500, 2032), (5, 16384), (4, 16400), (2, 70000)])
def test_quantizer_is_exact(rows, K, dtype):
    rng = np.random.default_rng(rows + K)
    x = values(rng, (rows, K), dtype, 1.0) * torch.exp(2 * torch.randn(rows, 1, device="cuda")).to(dtype)
    q, s = mq.quantize_int8_rows(x)
    rq, rs = oracle.quantize_int8(host(x).astype(np.float32))
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)


def test_quantizer_edges():
    tiny = 2.0 ** -120
    rows = [[0.0] * 32, [tiny * 0.75] + [0.0] * 31, [tiny] + [-tiny / 3] * 31, [3.0e38] + [1.0e38] * 31,
            [-1.0] + [0.5 / 127] * 31, [127.0] + [0.5, 1.5, 2.5, -0.5, -1.5] + [0.0] * 26,
            [float("inf")] + [1.0] * 31, [1.0] * 31 + [float("nan")], [float("-inf"), float("nan")] + [0.0] * 30]
    x = torch.tensor(rows, dtype=F32, device="cuda")
    q, s = mq.quantize_int8_rows(x)
    rq, rs = oracle.quantize_int8(x.cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.cpu().numpy()[:6], rq[:6])
    # a row past the registers' length, its special value at either end
    for at in (0, 16399):
        x = torch.ones(2, 16400, dtype=BF16, device="cuda")
        x[1, at] = float("nan")
        q, s = mq.quantize_int8_rows(x)
        assert float(s[0]) == float(np.float32(1) / np.float32(127)) and bool(torch.isnan(s[1]))


def test_quantizer_past_the_infinity_cache():
    # 300 MB of f16: the variant that streams past the caches, compared in parts
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(10007, 15008, generator=g, device="cuda").to(F16)
    q, s = mq.quantize_int8_rows(x)
    for i in (0, 1, 5000, 10006):
        rq, rs = oracle.quantize_int8(host(x[i:i + 1]).astype(np.float32))
        assert np.array_equal(q[i:i + 1].cpu().numpy(), rq) and np.array_equal(s[i:i + 1].cpu().numpy(), rs)
    m = x.abs().amax(1).float()
    full = torch.full_like(m, 127.0)
    assert torch.equal(s, m / full)
    for lo in range(0, 10007, 1000):
        p = (x[lo:lo + 1000].float() * (full / m)[lo:lo + 1000, None]).round()
        assert torch.equal(q[lo:lo + 1000], p.to(torch.int8))


# --------------------------------------------------------------------- GEMM
class Experts:
    def __init__(self, seed, T, k, E, N, K, a_row="token", kind="distinct", skip=0.0):
        rng, self.ids, (self.off, self.srt, self.p2s, _) = tables(seed, T, k, E, kind, skip)
        self.T, self.k, self.E, self.N, self.K, self.P, self.n = T, k, E, N, K, T * k, int(self.off[-1])
        self.a_row, self.rng = a_row, rng
        rows = T if a_row == "token" else self.P
        self.a = rng.integers(-128, 128, (rows, K)).astype(np.int8)
        self.w = rng.integers(-128, 128, (E, N, K)).astype(np.int8)
        self.sa = (rng.random(rows) + 0.5).astype(np.float32) / 64
        self.sw = ((rng.random((E, N)) + 0.5) * K ** -0.5 / 64).astype(np.float32)
        self.d = {n: dev(getattr(self, n)) for n in ("a", "w", "sa", "sw", "off", "srt")}

    def run(self, dtype, act="none", out=None, **kw):
        d = self.d
        kw = dict(dict(a_row=self.a_row), **kw)
        return mq.grouped_gemm_qint8(d["a"], d["sa"], d["w"], d["sw"], d["off"], d["srt"], self.k, act=act,
                                     out_dtype=dtype, out=out, **kw)

    def oracle(self):
        return oracle.grouped_gemm_qint8(self.a, self.sa, self.a_row, self.w, self.sw, self.off, self.srt, self.k)


GEMMS = [  # T, k, E, N, K, a_row, kind, skip
    (1, 1, 1, 32, 128, "token", "distinct", 0.0),
    (1, 8, 256, 64, 256, "token", "distinct", 0.0),
    (8, 8, 64, 512, 1152, "token", "distinct", 0.0),
    (9, 1, 1, 288, 384, "sorted", "one", 0.0),                # nine rows: one more than a wave's item
    (17, 3, 5, 96, 128, "token", "repeat", 0.3),
    (64, 2, 4, 256, 256, "token", "distinct", 0.0),
    (64, 2, 4, 256, 256, "token", "none", 0.0),
    (63, 1, 1, 544, 128, "sorted", "one", 0.0),               # rows around the tiles' heights
    (65, 1, 1, 480, 640, "token", "one", 0.0),
    (127, 1, 1, 32, 128, "token", "one", 0.0),
    (129, 1, 2, 1056, 384, "token", "one", 0.0),
    (257, 1, 1, 800, 256, "sorted", "one", 0.0),
    (301, 3, 37, 1056, 1152, "sorted", "repeat", 0.2),
    (40, 2, 1024, 64, 128, "token", "repeat", 0.1),           # the most experts
    (700, 2, 7, 320, 512, "token", "repeat", 0.1),
    (900, 4, 9, 1312, 896, "token", "distinct", 0.05),
]
GIDS = [f"T{c[0]}k{c[1]}E{c[2]}N{c[3]}K{c[4]}-{c[5]}-{c[6]}" for c in GEMMS]


@pytest.mark.parametrize("case", GEMMS, ids=GIDS)
def test_gemm_every_type_and_schedule(case):
    p = Experts(11, *case)
    r = p.oracle()
    n, I = p.n, p.N // 2
    seen = {}
    for sched in ("auto", "decode", "prefill"):
        out = torch.full((p.P, p.N), 77, dtype=torch.int32, device="cuda")
        assert p.run(torch.int32, out=out, sched=sched) is out
        assert np.array_equal(out[:n].cpu().numpy(), r["acc"]), sched
        assert bool((out[n:] == 77).all())                    # rows of no expert stay as they were
        for dtype in (F16, BF16, F32):
            y = host(p.run(dtype, sched=sched))[:n]
            within(y, r["y"], half_step(r["y"], dtype) + 4 * U * np.abs(r["y"]), (sched, dtype))
            out = torch.full((p.P, I), 7.0, dtype=dtype, device="cuda")
            h = host(p.run(dtype, act="silu_mul", out=out, sched=sched))
            ref, g = oracle.silu_gate(r["y"]), np.abs(r["y"][:, :I])
            within(h[:n], ref, half_step(ref, dtype) + (16 + 8 * g) * U * np.abs(ref) + 2.0 ** -118, (sched, dtype, "silu"))
            assert np.all(h[n:] == 7)
            for x, v in (("y", y), ("h", h[:n])):             # every schedule gives the same bits
                assert np.array_equal(seen.setdefault((x, dtype), v), v), (sched, dtype, x)


def test_gemm_every_row_as_it_is():
    # no sorted_pair_ids: row s is row s; and P below a's rows
    p = Experts(12, 300, 1, 3, 288, 256, "sorted", "repeat")
    ref = p.run(torch.int32)
    d = p.d
    for a_row in ("token", "sorted"):
        got = mq.grouped_gemm_qint8(d["a"], d["sa"], d["w"], d["sw"], d["off"], None, 1, a_row=a_row, out_dtype=torch.int32)
        assert torch.equal(got, ref)
    more = torch.cat([d["a"], d["a"][:9]])
    got = mq.grouped_gemm_qint8(more, torch.cat([d["sa"], d["sa"][:9]]), d["w"], d["sw"], d["off"], d["srt"], 1,
                                a_row="sorted", out_dtype=torch.int32)
    assert torch.equal(got, ref)


@pytest.mark.parametrize("counts", [(1, 0, 9), (70, 3, 130), (300, 0, 500)])
@pytest.mark.parametrize("K", [128, 256, 1024, 1152, 4096])
def test_gemm_sums_that_start_anywhere(K, counts):
    # workgroups and waves start their sums over K at places of their own: enough of them for
    # every place, K of one stage and more, powers of two and not
    g = torch.Generator(device="cuda").manual_seed(K + counts[0])
    P, N, E = sum(counts), 4096, len(counts)
    code = lambda *s: torch.randint(-128, 128, s, dtype=torch.int8, device="cuda", generator=g)
    a, w = code(P, K), code(E, N, K)
    one = [torch.ones(s, device="cuda") for s in ((P,), (E, N))]
    ends = np.cumsum((0,) + counts)
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    # float64 products of integers below 2^53 are exact
    want = torch.cat([a[lo:hi].double() @ w[e].double().T.contiguous()
                      for e, (lo, hi) in enumerate(zip(ends, ends[1:]))]).int()
    for sched in ("decode", "prefill"):
        for _ in range(2):
            got = mq.grouped_gemm_qint8(a, one[0], w, one[1], off, None, 1, out_dtype=torch.int32, sched=sched)
            assert torch.equal(got, want), sched


def test_gemm_the_largest_sums_and_scales():
    # every code -128: the int32 sums' largest, K = 131072 - 128; and scales at the ends of fp32
    K, N, P = 131072 - 128, 64, 40
    a = torch.full((P, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((1, N, K), -128, dtype=torch.int8, device="cuda")
    w[0, 1::2] = 127
    off = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    sa = torch.full((P,), 2.0 ** -100, device="cuda")
    sw = torch.full((1, N), 2.0 ** 60, device="cuda")
    want = torch.tensor([128 * 128 * K, -128 * 127 * K], device="cuda").repeat(N // 2)
    for sched in ("decode", "prefill"):
        acc = mq.grouped_gemm_qint8(a, sa, w, sw, off, None, 1, out_dtype=torch.int32, sched=sched)
        assert torch.equal(acc.long(), want.expand(P, N))
        y = mq.grouped_gemm_qint8(a, sa, w, sw, off, None, 1, out_dtype=F32, sched=sched)
        assert torch.equal(y, (want.double() * 2.0 ** -40).float().expand(P, N))
    sa[3] = float("nan")                                       # a row that the quantizer could not represent
    y = mq.grouped_gemm_qint8(a, sa, w, sw, off, None, 1, out_dtype=F32)
    assert bool(torch.isnan(y[3]).all()) and not bool(torch.isnan(y[:3]).any()) and not bool(torch.isnan(y[4:]).any())


def test_gemm_offsets_past_32_bits():
    """300 experts of 2048 x 8192: 5 GB of weights, and an output of more than
    2^32 bytes; the last rows and experts against sums of their own."""
    E, N, K = 300, 2048, 8192
    g = torch.Generator(device="cuda").manual_seed(13)
    w = torch.randint(-128, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand(E, N, generator=g, device="cuda") + 0.5
    P = 540000                                                 # x 2048 x 4 bytes = 4.4 GB
    off = torch.full((E + 1,), P, dtype=torch.int32)
    off[0], off[1:E] = 0, P - 50
    off = off.cuda()
    a = torch.randint(-128, 128, (P, 128), generator=g, device="cuda", dtype=torch.int8)
    y = mq.grouped_gemm_qint8(a, torch.ones(P, device="cuda"), w[:, :, :128].contiguous(), sw, off, None, 1,
                              out_dtype=torch.int32)
    for rows, e in ((slice(P - 100, P - 50), 0), (slice(P - 50, P), E - 1)):
        assert torch.equal(y[rows].double(), a[rows].double() @ w[e, :, :128].double().T)
    del y, a
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[E - 1], off[E] = 3, 8                                  # 3 rows of expert E - 2, 5 of the last
    a = torch.randint(-128, 128, (8, K), generator=g, device="cuda", dtype=torch.int8)
    dy = torch.randn(8, N, generator=g, device="cuda").to(BF16)
    for sched in ("decode", "prefill"):
        y = mq.grouped_gemm_qint8(a, torch.ones(8, device="cuda"), w, sw, off.cuda(), None, 1, out_dtype=torch.int32,
                                  sched=sched)
        for rows, e in ((slice(0, 3), E - 2), (slice(3, 8), E - 1)):
            assert torch.equal(y[rows].double(), a[rows].double() @ w[e].double().T)
    dx = mq.grouped_gemm_qint8_backward(dy, w, sw, off.cuda())
    for rows, e in ((slice(0, 3), E - 2), (slice(3, 8), E - 1)):
        d = dy[rows].double() * sw[e].double()
        ref, m = d @ w[e].double(), d.abs().amax(1, keepdim=True)
        tol = half_step(host(ref.float()), BF16) + host((0.51 / 32512 * m * w[e].double().abs().sum(0) +
                                                          8 * U * (d.abs() @ w[e].double().abs())).float())
        within(host(dx[rows]), ref.cpu().numpy(), tol)


# Rows of an expert around every tile's height and its halves and quarters; few
# experts with many rows.  With these widths each tile size of the schedule is
# the one taken (64 x 128, 64, 128 and 256 x 256).
MANY = [0, 1, 15, 16, 17, 31, 33, 47, 64, 65, 100, 128, 129, 200, 255, 256, 257, 300, 511, 513, 0, 77]
FEW = [3000, 257, 1100]


def grouped(counts, N, K, seed=14, rows_past=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    n, E = int(off[-1]), len(counts)
    a = torch.randint(-128, 128, (n + rows_past, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    sa = (torch.rand(n + rows_past, generator=g, device="cuda") + 0.5) / 64
    sw = (torch.rand(E, N, generator=g, device="cuda") + 0.5) * K ** -0.5 / 64
    return g, off, off.tolist(), n, a, w, sa, sw


@pytest.mark.parametrize("counts,N,K", [(MANY, 288, 128), (MANY, 1024, 384), (MANY, 4096, 256), (FEW, 4096, 256),
                                        (FEW, 4352, 128)])
def test_gemm_tiles_of_every_height(counts, N, K):
    g, off, at, n, a, w, sa, sw = grouped(counts, N, K)
    order = torch.cat([torch.randperm(n, generator=g, device="cuda"), torch.full((5,), -1, device="cuda")]).int()
    I = N // 2
    for srt, topk, a_row in ((None, 1, "sorted"), (order, 1, "token")):
        acc = torch.full((n + 5, N), 77, dtype=torch.int32, device="cuda")
        mq.grouped_gemm_qint8(a, sa, w, sw, off, srt, topk, a_row=a_row, out_dtype=torch.int32, out=acc, sched="prefill")
        h = torch.full((n + 5, I), 7.0, device="cuda")
        mq.grouped_gemm_qint8(a, sa, w, sw, off, srt, topk, a_row=a_row, act="silu_mul", out_dtype=F32, out=h,
                              sched="prefill")
        row = torch.arange(n, device="cuda") if srt is None else srt[:n].long()
        for e, (lo, hi) in enumerate(zip(at, at[1:])):
            if hi == lo:
                continue
            r = row[lo:hi]
            ref = a[r].double() @ w[e].double().T.contiguous()
            assert torch.equal(acc[lo:hi].double(), ref), (a_row, e)
            y = ref * sa[r].double()[:, None] * sw[e].double()
            ref = y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:]
            tol = (16 + 8 * y[:, :I].abs()) * U * ref.abs() + U * ref.abs() + 2.0 ** -118
            assert bool(((h[lo:hi].double() - ref).abs() <= tol).all()), (a_row, e)
        assert bool((acc[n:] == 77).all()) and bool((h[n:] == 7).all())


@pytest.mark.parametrize("counts,N,K", [(MANY, 160, 128), (MANY, 96, 512), (MANY, 288, 2048), (MANY, 128, 1920),
                                        (FEW, 224, 2048), (FEW, 128, 2176)])
def test_gradient_tiles_of_every_height(counts, N, K):
    g, off, at, n, _, w, _, sw = grouped(counts, N, K, 15)
    dy = torch.randn(n + 5, N, generator=g, device="cuda").to(BF16)
    base = torch.randn(n + 5, K, generator=g, device="cuda").to(BF16)
    dx = torch.full((n + 5, K), 7.0, dtype=BF16, device="cuda")
    mq.grouped_gemm_qint8_backward(dy, w, sw, off, base=base, dx=dx)
    for e, (lo, hi) in enumerate(zip(at, at[1:])):
        if hi == lo:
            continue
        d, we = dy[lo:hi].double() * sw[e].double(), w[e].double()
        ref = d @ we + base[lo:hi].double()
        tol = (ref.abs() * 2.0 ** -8 + 0.51 / 32512 * d.abs().amax(1, keepdim=True) * we.abs().sum(0) +
               8 * U * (d.abs() @ we.abs()) + U * base[lo:hi].double().abs() + 1e-40)
        assert bool(((dx[lo:hi].double() - ref).abs() <= tol).all()), e
    assert bool((dx[n:] == 7).all())
    # a row's bits do not depend on the rows beside it, which choose the tile
    lo, hi = at[-2], at[-2] + 3
    one = torch.zeros_like(off)
    one[-1] = 3
    alone = mq.grouped_gemm_qint8_backward(dy[lo:hi].clone(), w, sw, one, base=base[lo:hi].clone())
    assert torch.equal(alone, dx[lo:hi])


# ----------------------------------------------------------------- gradient
GRADS = [  # T, k, E, N, K, kind, skip
    (1, 1, 1, 32, 128, "distinct", 0.0),
    (1, 8, 256, 64, 128, "distinct", 0.0),
    (17, 3, 5, 96, 128, "repeat", 0.3),
    (31, 1, 1, 160, 384, "one", 0.0),
    (33, 1, 1, 64, 640, "one", 0.0),
    (64, 2, 4, 256, 256, "distinct", 0.0),
    (64, 2, 4, 256, 256, "none", 0.0),
    (63, 1, 2, 288, 896, "one", 0.0),
    (65, 1, 1, 1056, 256, "one", 0.0),
    (128, 1, 1, 96, 1152, "one", 0.0),
    (301, 3, 37, 544, 1152, "repeat", 0.2),
    (40, 2, 1024, 64, 128, "repeat", 0.1),
    (700, 2, 7, 2080, 384, "repeat", 0.1),
    (900, 4, 9, 8224, 128, "distinct", 0.05),
    (20, 2, 3, 32800, 256, "repeat", 0.1),                    # rows longer than the registers hold
]


def grad_case(p, dtype, base, dy=None):
    dy = values(p.rng, (p.P, p.N), dtype, 0.1) if dy is None else dy
    dy[p.n:] = float("nan")                                   # rows of no expert are not read
    b = values(p.rng, (p.P, p.K), dtype) if base else None
    return dy, b


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("case", GRADS, ids=[f"T{c[0]}k{c[1]}E{c[2]}N{c[3]}K{c[4]}-{c[5]}" for c in GRADS])
def test_gradient(case, dtype):
    T, k, E, N, K, kind, skip = case
    p = Experts(21, T, k, E, N, K, "sorted", kind, skip)
    n = p.n
    for base in (False, True):
        dy, b = grad_case(p, dtype, base)
        r = oracle.grouped_gemm_qint8_backward(np.nan_to_num(host(dy)), p.w, p.sw, p.off, host(b) if base else None)
        tol = (half_step(r["dx"], dtype) + 0.51 / 32512 * r["top"][:, None] * r["wsum"] + 8 * U * r["mag"] +
               (U * np.abs(host(b)) if base else 0))
        dx = torch.full((p.P, K), 7.0, dtype=dtype, device="cuda")
        ws = torch.full((mq.qint8_backward_workspace_bytes(p.P, E, N, K),), 255, dtype=torch.uint8, device="cuda")
        assert mq.grouped_gemm_qint8_backward(dy, p.d["w"], p.d["sw"], p.d["off"], base=b, dx=dx, workspace=ws) is dx
        within(host(dx)[:n], r["dx"][:n], tol[:n], base)
        assert np.all(host(dx)[n:] == 7)
        again = mq.grouped_gemm_qint8_backward(dy, p.d["w"], p.d["sw"], p.d["off"], base=b)
        assert torch.equal(again[:n], dx[:n])                 # equal inputs, equal bits; the workspace's old contents unread
        if base:                                              # in place
            got = mq.grouped_gemm_qint8_backward(dy, p.d["w"], p.d["sw"], p.d["off"], base=b, dx=b)
            assert got is b and torch.equal(b[:n], dx[:n])


def test_gradient_against_differences_of_the_product():
    """<dx, x> moves as the forward call's <dy, y> does: with activations whose
    codes are exact (whole numbers times a power of two), the difference of two
    products is the gradient's."""
    p = Experts(22, 40, 1, 3, 96, 256, "sorted", "repeat")
    dy, _ = grad_case(p, BF16, False)
    one = torch.full((p.P,), 0.5, device="cuda")
    a, b = (torch.randint(-128, 128, (p.P, p.K), device="cuda", dtype=torch.int8) for _ in range(2))
    y = [mq.grouped_gemm_qint8(v, one, p.d["w"], p.d["sw"], p.d["off"], p.d["srt"], 1, a_row="sorted", out_dtype=F32).double()
         for v in (a, b)]
    n = p.n
    diff = float((dy[:n].double() * (y[0] - y[1])[:n]).sum())
    dx = mq.grouped_gemm_qint8_backward(dy, p.d["w"], p.d["sw"], p.d["off"])
    step = (a.double() - b.double())[:n] * 0.5
    got = float((dx[:n].double() * step).sum())
    r = oracle.grouped_gemm_qint8_backward(np.nan_to_num(host(dy)), p.w, p.sw, p.off)
    tol = half_step(r["dx"], BF16) + 0.51 / 32512 * r["top"][:, None] * r["wsum"] + 8 * U * r["mag"]
    room = float((torch.from_numpy(tol[:n]).cuda() * step.abs()).sum())
    assert abs(got - diff) <= room + 4 * U * float((dy[:n].double().abs() * (y[0].abs() + y[1].abs())[:n]).sum())


def test_gradient_rows_of_every_kind():
    """Zeros, one value alone, values far apart, rows below 2^-100, infinities
    and NaN: each row by itself, the others untouched by it."""
    N, K, P = 160, 256, 70
    rng = np.random.default_rng(23)
    w = rng.integers(-128, 128, (1, N, K)).astype(np.int8)
    sw = np.exp(2 * rng.standard_normal((1, N))).astype(np.float32)
    dy = rng.standard_normal((P, N)) * 0.1
    dy[0] = 0
    dy[1] = 0
    dy[1, 159] = 3.0
    dy[2] *= np.exp(12 * rng.random(N))
    dy[3] *= 2.0 ** -115
    dy[4] *= 2.0 ** 100
    t = torch.from_numpy(dy).to(BF16).cuda()
    t[65, 0], t[66, 159], t[67, 3] = float("inf"), float("nan"), float("-inf")
    off = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    dx = host(mq.grouped_gemm_qint8_backward(t, dev(w), dev(sw), off))
    assert np.isnan(dx[[65, 66, 67]]).all() and not dx[0].any() and not dx[3].any()
    keep = np.r_[0:3, 4:65, 68:70]
    r = oracle.grouped_gemm_qint8_backward(host(t)[keep], w, sw, np.array([0, keep.size]))
    within(dx[keep], r["dx"], half_step(r["dx"], BF16) + 0.51 / 32512 * r["top"][:, None] * r["wsum"] + 8 * U * r["mag"])


# --------------------------------------------------------------- activation
def silu_tol(gu, dtype):
    I = gu.shape[1] // 2
    ref = oracle.silu_gate(gu)
    return ref, half_step(ref, dtype) + (16 + 8 * np.abs(gu[:, :I])) * U * np.abs(ref) + 2.0 ** -118 * (1 + np.abs(gu[:, I:]))


def grad_tol(dh, gu, dtype):
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    ref = oracle.silu_gate_backward(dh, gu)
    s, c = (1 / (1 + np.exp(-np.clip(v, -700, 700))) for v in (g, -g))
    a, b = np.abs(dh * u), np.abs(dh)
    t = np.abs(g * s)
    tol = np.concatenate([(16 + 4 * np.abs(g)) * U * a * (s + t * c) + 4 * U * a * t + 2.0 ** -118 * (a + 1),
                          (16 + 8 * np.abs(g)) * U * b * t + 2.0 ** -118 * (b + 1)], axis=1)
    return ref, half_step(ref, dtype) + tol


SILUS = [  # P, I, last expert's end (None: no offsets)
    (1, 8, None), (5, 8, 3), (7, 128, 7), (33, 136, 20), (64, 1000, 50), (300, 2048, 300), (41, 2056, 0), (9, 14336, None),
    (1000, 24, 999),
]


def silu_inputs(P, I, dtype):
    rng = np.random.default_rng(P + I)
    gu = values(rng, (P, 2 * I), dtype, 3.0)
    gu[0, 0], gu[0, I - 1] = 60.0, -60.0
    return rng, gu


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("P,I,end", SILUS)
def test_silu_and_gradient(P, I, end, dtype):
    rng, gu = silu_inputs(P, I, dtype)
    n, B = P if end is None else end, -(-I // 128)
    off = None if end is None else torch.tensor([0, end // 2, end], dtype=torch.int32, device="cuda")
    gu[n:] = float("nan")
    h = torch.full((P, I), 7.0, dtype=dtype, device="cuda")
    assert mq.moe_silu_mul(gu, off, h=h)[1:] == (None, None)
    v = host(gu)[:n]
    ref, tol = silu_tol(v, dtype)
    within(host(h)[:n], ref, tol, "h")
    assert np.all(host(h)[n:] == 7)
    ck = torch.full((P, 2 * I), 77, dtype=torch.int8, device="cuda")
    cs = torch.full((P, 2 * B), 7.0, device="cuda")
    h2, *_ = mq.moe_silu_mul(gu, off, checkpoint=True, ck=ck, cs=cs)
    assert torch.equal(h2[:n], h[:n])
    rck, rcs = oracle.checkpoint(v.astype(np.float32))
    assert np.array_equal(ck[:n].cpu().numpy(), rck) and np.array_equal(cs[:n].cpu().numpy(), rcs)
    assert bool((ck[n:] == 77).all()) and bool((cs[n:] == 7).all())

    dh = values(rng, (P, I), dtype)
    dh[n:] = float("nan")
    kept = oracle.checkpoint_values(rck, rcs)
    for kw, val in ((dict(gu=gu), v), (dict(ck=ck, cs=cs), kept)):
        dgu = torch.full((P, 2 * I), 7.0, dtype=dtype, device="cuda")
        assert mq.moe_silu_mul_backward(dh, off, dgu=dgu, **kw)[1] is None
        ref, tol = grad_tol(host(dh)[:n], val, dtype)
        within(host(dgu)[:n], ref, tol, "dgu")
        h = torch.full((P, I), 7.0, dtype=dtype, device="cuda")
        d2, got = mq.moe_silu_mul_backward(dh, off, need_h=True, h=h, **kw)
        assert got is h and torch.equal(d2[:n], dgu[:n])
        ref, tol = silu_tol(val, dtype)
        within(host(h)[:n], ref, tol, "h again")
        assert np.all(host(h)[n:] == 7) and np.all(host(dgu)[n:] == 7)
    again = torch.full((P, I), 7.0, dtype=dtype, device="cuda")
    assert mq.moe_silu_mul_again(ck, cs, off, dtype=dtype, h=again) is again and torch.equal(again, h)
    inplace = gu.clone()
    assert mq.moe_silu_mul_backward(dh, off, gu=inplace, dgu=inplace)[0] is inplace
    assert torch.equal(inplace[:n], mq.moe_silu_mul_backward(dh, off, gu=gu)[0][:n])
    assert bool(torch.isnan(inplace[n:]).all())


def test_silu_far_values_infinities_and_nan():
    I = 136
    gu = torch.ones(8, 2 * I, dtype=F32, device="cuda")
    gu[0, :4] = torch.tensor([200.0, -200.0, 3.0e38, -3.0e38])
    gu[1, 0], gu[2, I + 5], gu[3, 130], gu[4, 2 * I - 1] = float("inf"), float("nan"), float("-inf"), float("inf")
    h, ck, cs = mq.moe_silu_mul(gu, checkpoint=True)
    assert h[0, :4].tolist() == [200.0, 0.0, float(torch.tensor(3.0e38)), 0.0]
    # a block's scale shows what it held, the other blocks are as ever
    bad = torch.zeros(8, 4, dtype=torch.bool)
    bad[1, 0] = bad[2, 2] = bad[3, 1] = bad[4, 3] = True
    assert torch.equal(torch.isnan(cs).cpu(), bad)
    dh = torch.ones(8, I, dtype=F32, device="cuda")
    d = mq.moe_silu_mul_backward(dh, gu=gu)[0]
    assert d[0, :4].tolist() == [1.0, 0.0, 1.0, 0.0] and d[0, I:I + 2].tolist() == [200.0, 0.0]
    k = mq.moe_silu_mul_backward(dh, ck=ck, cs=cs)[0].cpu()
    nan = torch.isnan(k)
    assert nan[1, :128].all() and nan[1, I:I + 128].all() and not nan[1, 128:I].any() and not nan[1, I + 128:].any()
    assert nan[2, :128].all() and not nan[2, I:].any()         # an unknown up: the gate's gradient alone
    assert nan[4, 128:I].all() and not nan[0].any() and not nan[5:].any()


def test_silu_past_the_infinity_cache():
    # streams of more than 256 MB and rows past 2^32 bytes: the last rows against themselves alone
    P, I = 40000, 14344
    g = torch.Generator(device="cuda").manual_seed(31)
    gu = torch.empty(P, 2 * I, dtype=F32, device="cuda").normal_(generator=g)
    dh = torch.empty(P, I, dtype=F32, device="cuda").normal_(generator=g)
    h, ck, cs = mq.moe_silu_mul(gu, checkpoint=True)
    dgu, h2 = mq.moe_silu_mul_backward(dh, ck=ck, cs=cs, need_h=True)
    d2 = mq.moe_silu_mul_backward(dh, gu=gu)[0]
    for rows in (slice(0, 3), slice(P - 5, P)):
        a, b = gu[rows].clone(), dh[rows].clone()
        rh, rck, rcs = mq.moe_silu_mul(a, checkpoint=True)
        assert torch.equal(h[rows], rh) and torch.equal(ck[rows], rck) and torch.equal(cs[rows], rcs)
        rd, rh2 = mq.moe_silu_mul_backward(b, ck=rck, cs=rcs, need_h=True)
        assert torch.equal(dgu[rows], rd) and torch.equal(h2[rows], rh2)
        assert torch.equal(d2[rows], mq.moe_silu_mul_backward(b, gu=a)[0])


# ----------------------------------------------------- together, as they run
def _layer(T=96, k=2, E=5, H=256, I=256, R=16, dtype=BF16, seed=41):
    """A layer of frozen INT8 experts with adapters beside both projections."""
    rng, _, route = tables(seed, T, k, E, "repeat", 0.1)
    P = T * k
    q = dict(k=k, E=E, H=H, I=I, R=R, P=P, dtype=dtype, off=dev(route[0]), srt=dev(route[1]), p2s=dev(route[2]),
             tw=dev((rng.random((T, k)) + 0.1).astype(np.float32)), x=values(rng, (T, H), dtype),
             dout=values(rng, (T, H), dtype, 0.1), scale=dev((rng.random(E) + 0.5).astype(np.float32)))
    for name, (n, m) in (("1", (2 * I, H)), ("2", (H, I))):
        q["w" + name] = dev(np.clip(np.rint(32 * rng.standard_normal((E, n, m))), -127, 127).astype(np.int8))
        q["s" + name] = dev(((rng.random((E, n)) + 0.5) * m ** -0.5 / 32).astype(np.float32))
        q["a" + name] = values(rng, (E, R, m), dtype, m ** -0.5)
        q["b" + name] = values(rng, (E, n, R), dtype, R ** -0.5)
    z = lambda *s, dt=dtype: torch.zeros(*s, dtype=dt, device="cuda")
    i8, f4 = torch.int8, torch.float32
    b = dict(xq=z(T, H, dt=i8), xs=z(T, dt=f4), gu=z(P, 2 * I), hl1=z(P, R, dt=f4), h=z(P, I), ck=z(P, 2 * I, dt=i8),
             cs=z(P, 2 * -(-I // 128), dt=f4), hq=z(P, I, dt=i8), hs=z(P, dt=f4), y=z(P, H), hl2=z(P, R, dt=f4), out=z(T, H),
             dy=z(P, H), dw=z(T, k, dt=f4), dh=z(P, I), da2=z(E, R, I), db2=z(E, H, R), dgu=z(P, 2 * I), h2=z(P, I),
             da1=z(E, R, H), db1=z(E, 2 * I, R), dxs=z(P, H), dx=z(T, H))
    u8 = lambda n: torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
    ws = dict(f1=u8(mq.lora_workspace_bytes(P, E, 2 * I, H, R)), f2=u8(mq.lora_workspace_bytes(P, E, H, I, R)),
              b1=u8(mq.lora_workspace_bytes(P, E, 2 * I, H, R, backward=True)),
              b2=u8(mq.lora_workspace_bytes(P, E, H, I, R, backward=True)),
              g1=u8(mq.qint8_backward_workspace_bytes(P, E, 2 * I, H)), g2=u8(mq.qint8_backward_workspace_bytes(P, E, H, I)))
    return q, b, ws


def _train(q, b, ws):
    """Forward and backward of one layer: only the 8-bit checkpoint and the
    low-rank values are kept of what lies between x and out."""
    o, s, p, k, sc = q["off"], q["srt"], q["p2s"], q["k"], q["scale"]
    mq.quantize_int8_rows(q["x"], q=b["xq"], scale=b["xs"])
    mq.grouped_gemm_qint8(b["xq"], b["xs"], q["w1"], q["s1"], o, s, k, out_dtype=q["dtype"], out=b["gu"])
    mq.grouped_lora(q["x"], q["a1"], q["b1"], o, s, k, base=b["gu"], out=b["gu"], h=b["hl1"], scale=sc, workspace=ws["f1"])
    mq.moe_silu_mul(b["gu"], o, checkpoint=True, h=b["h"], ck=b["ck"], cs=b["cs"])
    mq.quantize_int8_rows(b["h"], q=b["hq"], scale=b["hs"])
    mq.grouped_gemm_qint8(b["hq"], b["hs"], q["w2"], q["s2"], o, s, k, a_row="sorted", out_dtype=q["dtype"], out=b["y"])
    mq.grouped_lora(b["h"], q["a2"], q["b2"], o, s, k, a_row="sorted", base=b["y"], out=b["y"], h=b["hl2"], scale=sc,
                    workspace=ws["f2"])
    mq.moe_scatter_combine(b["y"], p, q["tw"], out=b["out"])

    mq.moe_scatter_combine_backward(q["dout"], b["y"], p, q["tw"], dy=b["dy"], dw=b["dw"])
    # the adapters' part of dh, from h made again, then the frozen product's added to it in place
    mq.moe_silu_mul_again(b["ck"], b["cs"], o, dtype=q["dtype"], h=b["h2"])
    mq.grouped_lora_backward(b["dy"], b["h2"], q["a2"], q["b2"], b["hl2"], o, s, k, scale=sc, a_row="sorted", dx=b["dh"],
                             da=b["da2"], db=b["db2"], workspace=ws["b2"])
    mq.grouped_gemm_qint8_backward(b["dy"], q["w2"], q["s2"], o, base=b["dh"], dx=b["dh"], workspace=ws["g2"])
    mq.moe_silu_mul_backward(b["dh"], o, ck=b["ck"], cs=b["cs"], dgu=b["dgu"])
    mq.grouped_lora_backward(b["dgu"], q["x"], q["a1"], q["b1"], b["hl1"], o, s, k, scale=sc, dx=b["dxs"], da=b["da1"],
                             db=b["db1"], workspace=ws["b1"])
    mq.grouped_gemm_qint8_backward(b["dgu"], q["w1"], q["s1"], o, base=b["dxs"], dx=b["dxs"], workspace=ws["g1"])
    mq.moe_permute_backward(b["dxs"], p, k, out=b["dx"])


def test_training_step_of_adapters_beside_int8_experts():
    """Every new step checked from the stored input of that step, so that no
    tolerance spans two roundings."""
    q, b, ws = _layer()
    _train(q, b, ws)
    off, srt, k, dt = host(q["off"]), host(q["srt"]), q["k"], q["dtype"]
    n = int(off[-1])
    xq, xs = oracle.quantize_int8(host(q["x"]).astype(np.float32))
    assert np.array_equal(b["xq"].cpu().numpy(), xq) and np.array_equal(host(b["xs"]).astype(np.float32), xs)
    gu = host(b["gu"])[:n]
    g0 = oracle.grouped_gemm_qint8(xq, xs, "token", q["w1"].cpu().numpy(), host(q["s1"]), off, srt, k)["y"]
    f = oracle.grouped_lora(host(q["x"]), host(q["a1"]), host(q["b1"]), off, srt, k, scale=host(q["scale"]))
    ref = g0 + f["out"][:n]          # the product was rounded once before the adapters were added
    within(gu, ref, half_step(ref, dt) + half_step(g0, dt) * (1 + 2.0 ** -8) + 4 * U * np.abs(g0) +
           U * (4 * (np.sqrt(256) + np.sqrt(16)) + 40) * (f["mag"][:n] + np.abs(g0)), "gu")
    ref, tol = silu_tol(gu, dt)
    within(host(b["h"])[:n], ref, tol, "h")
    ck, cs = oracle.checkpoint(gu.astype(np.float32))
    assert np.array_equal(b["ck"][:n].cpu().numpy(), ck)
    kept = oracle.checkpoint_values(ck, cs)
    ref, tol = silu_tol(kept, dt)
    within(host(b["h2"])[:n], ref, tol, "h again")
    hq, hs = oracle.quantize_int8(host(b["h"]).astype(np.float32))
    assert np.array_equal(b["hq"][:n].cpu().numpy(), hq[:n])
    dh = host(b["dh"])[:n]
    ref, tol = grad_tol(dh, kept, dt)
    within(host(b["dgu"])[:n], ref, tol, "dgu")
    for name, dyn, w, sw, x, a, bb, hl, row in (("dh", "dy", "w2", "s2", "h2", "a2", "b2", "hl2", "sorted"),
                                                 ("dxs", "dgu", "w1", "s1", "x", "a1", "b1", "hl1", "token")):
        d = host(b[dyn])
        x = host(b[x] if x in b else q[x])
        g = oracle.grouped_gemm_qint8_backward(d, q[w].cpu().numpy(), host(q[sw]), off)
        lo = oracle.grouped_lora_backward(d, x, host(q[a]), host(q[bb]), host(b[hl]), off, srt, k, scale=host(q["scale"]),
                                          a_row=row)
        ref = (g["dx"] + lo["dx"])[:n]
        tol = (half_step(ref, dt) + half_step(lo["dx"][:n], dt) * (1 + 2.0 ** -8) +
               (0.51 / 32512 * g["top"][:, None] * g["wsum"] + 9 * U * g["mag"])[:n] +
               U * (4 * (np.sqrt(512) + np.sqrt(256) + np.sqrt(16)) + 40) * lo["mdx"][:n])
        within(host(b[name])[:n], ref, tol, name)
    ref = oracle.permute_backward(host(b["dxs"]), host(q["p2s"]), k)
    within(host(b["dx"]), ref, half_step(ref, dt) + 4 * U * oracle.permute_backward(np.abs(host(b["dxs"])), host(q["p2s"]), k))


@pytest.mark.parametrize("kw", [dict(), dict(T=700, E=3, H=384, I=328 - 72, dtype=F16)])
def test_training_step_captured_and_replayed(kw):
    from tests.test_gpu_graphs import _capture_and_replay
    q, b, ws = _layer(**kw)
    n = int(q["off"][-1])            # rows of no expert keep what they hold
    rows = [b[x][:n] for x in ("gu", "h", "ck", "cs", "hq", "y", "dy", "h2", "dh", "dgu", "dxs")]
    _capture_and_replay(lambda: _train(q, b, ws),
                        rows + [b[x] for x in ("out", "dw", "da1", "db1", "da2", "db2", "dx")])


@pytest.mark.parametrize("T", [8, 900])
def test_serving_step_captured_and_replayed(T):
    from tests.test_gpu_graphs import _capture_and_replay
    q, b, _ = _layer(T=T, E=6, dtype=F16)
    h = torch.zeros(q["P"], q["I"], dtype=F16, device="cuda")

    def step():
        mq.quantize_int8_rows(q["x"], q=b["xq"], scale=b["xs"])
        mq.grouped_gemm_qint8(b["xq"], b["xs"], q["w1"], q["s1"], q["off"], q["srt"], q["k"], act="silu_mul", out=h)
        mq.quantize_int8_rows(h, q=b["hq"], scale=b["hs"])
        mq.grouped_gemm_qint8(b["hq"], b["hs"], q["w2"], q["s2"], q["off"], q["srt"], q["k"], a_row="sorted", out=b["y"])
        mq.moe_scatter_combine(b["y"], q["p2s"], q["tw"], out=b["out"])
    n = int(q["off"][-1])
    _capture_and_replay(step, [h[:n], b["hq"][:n], b["hs"][:n], b["y"][:n], b["out"]])


def test_two_streams_at_once_with_their_own_workspaces():
    p = Experts(44, 600, 2, 6, 1056, 640, "sorted", "repeat")
    dy, b = grad_case(p, BF16, True)
    gu = values(p.rng, (p.P, 1056), BF16)
    dy[p.n:] = 0

    def calls():
        return (p.run(BF16, act="silu_mul"), p.run(torch.int32, sched="decode"),
                mq.grouped_gemm_qint8_backward(dy, p.d["w"], p.d["sw"], p.d["off"], base=b),
                *mq.moe_silu_mul(gu, checkpoint=True), *mq.quantize_int8_rows(dy))
    ref = calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append(calls())
        torch.cuda.synchronize()
        for g in got:
            for i, (v, r) in enumerate(zip(g, ref)):
                rows = p.n if i < 3 else v.shape[0]
                assert torch.equal(v[:rows], r[:rows])


def test_malformed_tables_touch_nothing_out_of_range():
    """Offsets that fall, end past P or are negative, and ids out of range: the
    rows computed are then whatever, but every access stays inside."""
    p = Experts(45, 40, 2, 4, 96, 256)
    dy, _ = grad_case(p, F16, False)
    gu = values(p.rng, (p.P, 96), F16)
    for off in ([0, 70, 20, 1000, 5000], [-5, 10, 9, 40, 2000000000], [0, 0, 0, 0, -7]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        srt = p.d["srt"].clone()
        srt[5], srt[17], srt[30] = -1, p.P, 2000000000
        for sched in ("decode", "prefill"):
            out = torch.zeros(p.P + 8, p.N, dtype=torch.int32, device="cuda")
            mq.grouped_gemm_qint8(p.d["a"], p.d["sa"], p.d["w"], p.d["sw"], o, srt, 2, out_dtype=torch.int32, out=out,
                                  sched=sched)
            assert bool((out[p.P:] == 0).all())
        mq.grouped_gemm_qint8_backward(dy, p.d["w"], p.d["sw"], o)
        mq.moe_silu_mul(gu, o, checkpoint=True)
    torch.cuda.synchronize()


def test_no_rows():
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")
    i4, i8 = torch.int32, torch.int8
    q, s = mq.quantize_int8_rows(z(0, 64))
    off, w, sw = z(4, dt=i4), z(3, 64, 128, dt=i8), z(3, 64, dt=F32)
    for sched in ("auto", "decode", "prefill"):
        y = mq.grouped_gemm_qint8(z(0, 128, dt=i8), z(0, dt=F32), w, sw, off, z(0, dt=i4), 2, sched=sched)
        assert y.shape == (0, 64)
    assert mq.grouped_gemm_qint8_backward(z(0, 64), w, sw, off, base=z(0, 128)).shape == (0, 128)
    h, ck, cs = mq.moe_silu_mul(z(0, 272), off, checkpoint=True)
    assert h.shape == (0, 136) and ck.shape == (0, 272) and cs.shape == (0, 4)
    d, h = mq.moe_silu_mul_backward(z(0, 136), ck=ck, cs=cs, need_h=True)
    assert d.shape == (0, 272) and h.shape == (0, 136)
    assert mq.moe_silu_mul_backward(z(0, 136), gu=z(0, 272))[0].shape == (0, 272)
    assert mq.moe_silu_mul_again(ck, cs).shape == (0, 136)
    torch.cuda.synchronize()
