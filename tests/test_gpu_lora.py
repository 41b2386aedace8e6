"""grouped_lora and its gradient against the float64 oracle.

Tolerances, per element: the output's one rounding, half a step (finfo.eps /
2 relative, plus half the smallest subnormal), and the fp32 arithmetic before
it.  A chain of n fp32 additions rounds n times, each by at most 2^-24 of a
partial sum, which never exceeds the sum of the products' magnitudes (mag, from
the oracle); the roundings are independent, so 4 sqrt(n) of them bound their
sum.  A second 2^-24 per product covers the fp32 values split into 16-bit
parts, with 32 steps of room for the scale, the base and joining partial sums:
  tol = half step + 2^-24 (4 (sqrt K + sqrt N + sqrt R + sqrt P) + 32) mag."""
import numpy as np
import pytest
import torch

import oracle
import synth
from tests.gpu_util import dev, host
from tests.test_gpu_permute import BF16, F16, F32, half_step, tables, values

pytestmark = pytest.mark.gpu

mq = pytest.importorskip("quantized_moe_grouped_route_amd")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mq.lib()


def close(got, ref, mag, dtype, n, what, floor=0.0):
    tol = half_step(ref, dtype) + 2.0 ** -24 * (4 * sum(np.sqrt(v) for v in n) + 32) * mag + floor
    over = np.isinf(got) & (np.sign(got) == np.sign(ref)) & (np.abs(ref) + tol >= torch.finfo(dtype).max)
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - ref) <= tol) & ~over
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           float(np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300))))


class Problem:
    def __init__(self, seed, T, k, E, N, K, R, dtype, a_row="token", out_row="sorted", kind="distinct", skip=0.0,
                 scale=True):
        rng, self.ids, (self.off, self.srt, self.p2s, _) = tables(seed, T, k, E, kind, skip)
        self.T, self.k, self.E, self.N, self.K, self.R, self.dtype = T, k, E, N, K, R, dtype
        self.P, self.n = T * k, int(self.off[-1])
        self.kw = dict(a_row=a_row, out_row=out_row)
        self.x = values(rng, (T if a_row == "token" else self.P, K), dtype)
        if a_row == "sorted":
            self.x[self.n:] = float("nan")     # rows of no group are not read
        self.a = values(rng, (E, R, K), dtype, K ** -0.5)
        self.b = values(rng, (E, N, R), dtype, R ** -0.5)
        self.base = values(rng, (self.P, N), dtype)
        self.dy = values(rng, (self.P, N), dtype, 0.1)
        if out_row == "sorted":
            self.dy[self.n:] = float("nan")
        else:
            self.dy[torch.from_numpy(self.p2s < 0).cuda()] = float("nan")
        self.scale = (rng.random(E) + 0.25).astype(np.float32) if scale else None
        self.doff, self.dsrt, self.dp2s = dev(self.off), dev(self.srt), dev(self.p2s)
        self.dscale = dev(self.scale) if scale else None
        self.len = (K, N, R, self.P + 1)

    def forward(self, **kw):
        kw = dict(dict(base=self.base, scale=self.dscale, pair_to_sorted=self.dp2s, **self.kw), **kw)
        return mq.grouped_lora(self.x, self.a, self.b, self.doff, self.dsrt, self.k, **kw)

    def backward(self, h, **kw):
        return mq.grouped_lora_backward(self.dy, self.x, self.a, self.b, h, self.doff, self.dsrt, self.k,
                                        scale=self.dscale, **self.kw, **kw)

    def oracle(self, base="base"):
        x = np.nan_to_num(host(self.x))
        return oracle.grouped_lora(x, host(self.a), host(self.b), self.off, self.srt, self.k,
                                   base=host(self.base) if base else None, scale=self.scale, **self.kw)

    def oracle_grad(self, h):
        return oracle.grouped_lora_backward(np.nan_to_num(host(self.dy)), np.nan_to_num(host(self.x)), host(self.a),
                                            host(self.b), h, self.off, self.srt, self.k, scale=self.scale, **self.kw)


CASES = [  # T, k, E, N, K, R, a_row, out_row, kind, skip
    (1, 1, 1, 8, 8, 8, "token", "pair", "distinct", 0.0),
    (1, 1, 8, 4096, 4096, 16, "token", "pair", "distinct", 0.0),
    (5, 1, 300, 264, 136, 24, "token", "pair", "repeat", 0.4),
    (37, 1, 32, 1024, 2056, 64, "token", "pair", "repeat", 0.2),
    (8, 8, 256, 512, 1024, 16, "token", "sorted", "distinct", 0.0),
    (64, 2, 4, 256, 256, 8, "token", "sorted", "distinct", 0.0),
    (50, 3, 7, 72, 200, 40, "sorted", "sorted", "repeat", 0.3),
    (50, 3, 7, 72, 200, 40, "sorted", "pair", "repeat", 0.3),
    (33, 2, 5, 128, 128, 256, "token", "sorted", "distinct", 0.0),
    (20, 2, 1024, 40, 64, 136, "token", "pair", "repeat", 0.1),
    (64, 2, 4, 136, 264, 16, "token", "pair", "none", 0.0),
    (700, 2, 3, 392, 520, 32, "token", "sorted", "one", 0.0),
    (2100, 1, 2, 1032, 248, 16, "sorted", "sorted", "repeat", 0.05),
    (900, 4, 24, 520, 640, 72, "token", "sorted", "distinct", 0.1),
    (5000, 1, 3, 64, 72, 128, "token", "pair", "repeat", 0.5),
]
IDS = [f"T{c[0]}k{c[1]}E{c[2]}N{c[3]}K{c[4]}R{c[5]}-{c[6]}-{c[7]}-{c[8]}" for c in CASES]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case, dtype):
    T, k, E, N, K, R, a_row, out_row, kind, skip = case
    p = Problem(21, T, k, E, N, K, R, dtype, a_row, out_row, kind, skip)
    ref = p.oracle()
    h = torch.full((p.P, R), 3.0, device="cuda")
    out = torch.full((p.P, N), 7.0, dtype=dtype, device="cuda")
    assert p.forward(out=out, h=h) is out
    got = host(out)
    if out_row == "sorted":
        assert np.all(got[~ref["written"]] == 7)
        got, r, m = got[:p.n], ref["out"][:p.n], ref["mag"][:p.n]
    else:
        assert np.array_equal(got[~ref["written"]], host(p.base)[~ref["written"]])
        r, m = ref["out"], ref["mag"]
    close(got, r, m, dtype, p.len, "out")
    mh = np.zeros((p.P, R))
    rx = np.where(p.srt >= 0, p.srt // k, 0) if a_row == "token" else np.arange(p.P)
    x = np.abs(np.nan_to_num(host(p.x)))
    for e in range(E):
        i = slice(p.off[e], p.off[e + 1])
        mh[i] = x[rx[i]] @ np.abs(host(p.a[e])).T
    close(host(h)[:p.n], ref["h"][:p.n], mh[:p.n], F32, p.len, "h")
    assert np.all(host(h)[p.n:] == 3)
    # without h, and in place: the same bits; rows without a group keep theirs
    assert torch.equal(p.forward(out=torch.full_like(out, 7.0)), out)
    y = p.base.clone()
    p.forward(base=y, out=y, pair_to_sorted=None)
    if out_row == "sorted":
        assert torch.equal(y[:p.n], out[:p.n]) and torch.equal(y[p.n:], p.base[p.n:])
    else:
        assert torch.equal(y, out)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case, dtype):
    T, k, E, N, K, R, a_row, out_row, kind, skip = case
    p = Problem(22, T, k, E, N, K, R, dtype, a_row, out_row, kind, skip)
    h = torch.full((p.P, R), float("nan"), device="cuda")
    p.forward(h=h)
    hh = np.nan_to_num(host(h))
    ref = p.oracle_grad(hh)
    dx = torch.full((p.P, K), 7.0, dtype=dtype, device="cuda")
    da, db = torch.full_like(p.a, 9.0), torch.full_like(p.b, 9.0)
    got = p.backward(h, dx=dx, da=da, db=db)
    assert got[0] is dx and got[1] is da and got[2] is db
    assert np.all(host(dx)[p.n:] == 7)
    close(host(dx)[:p.n], ref["dx"][:p.n], ref["mdx"][:p.n], dtype, p.len, "dx")
    close(host(da), ref["da"], ref["mda"], dtype, p.len, "da")
    close(host(db), ref["db"], ref["mdb"], dtype, p.len, "db")
    empty = np.diff(p.off) == 0
    assert np.all(host(da)[empty] == 0) and np.all(host(db)[empty] == 0)
    # without dx, and again: the same bits
    none, da2, db2 = p.backward(h, need_dx=False)
    assert none is None and torch.equal(da, da2) and torch.equal(db, db2)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_no_base_and_no_scale(dtype):
    p = Problem(23, 30, 2, 6, 264, 520, 16, dtype, out_row="pair", kind="repeat", skip=0.3, scale=False)
    ref = p.oracle(base=None)
    got = host(p.forward(base=None))
    close(got, ref["out"], ref["mag"], dtype, p.len, "out")
    assert np.all(got[~ref["written"]] == 0)
    h = torch.zeros(p.P, 16, device="cuda")
    p.forward(h=h)
    g = p.oracle_grad(host(h))
    dx, da, db = p.backward(h)
    close(host(dx)[:p.n], g["dx"][:p.n], g["mdx"][:p.n], dtype, p.len, "dx")
    close(host(da), g["da"], g["mda"], dtype, p.len, "da")
    close(host(db), g["db"], g["mdb"], dtype, p.len, "db")


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_identity_rows_without_a_pair_table(dtype):
    rng = np.random.default_rng(24)
    off = np.array([0, 5, 5, 17, 40], np.int32)
    x, a, b = values(rng, (44, 72), dtype), values(rng, (4, 8, 72), dtype, 0.1), values(rng, (4, 136, 8), dtype)
    h = torch.zeros(44, 8, device="cuda")
    out = torch.full((44, 136), 7.0, dtype=dtype, device="cuda")
    mq.grouped_lora(x, a, b, dev(off), None, 1, a_row="sorted", out=out, h=h)
    ref = oracle.grouped_lora(host(x), host(a), host(b), off, None, 1, a_row="sorted", P=44)
    close(host(out)[:40], ref["out"][:40], ref["mag"][:40], dtype, (72, 136, 8, 44), "out")
    assert np.all(host(out)[40:] == 7)
    dy = values(rng, (44, 136), dtype)
    dx, da, db = mq.grouped_lora_backward(dy, x, a, b, h, dev(off), None, 1, a_row="sorted")
    g = oracle.grouped_lora_backward(host(dy), host(x), host(a), host(b), host(h), off, None, 1, a_row="sorted")
    close(host(dx)[:40], g["dx"][:40], g["mdx"][:40], dtype, (72, 136, 8, 44), "dx")
    close(host(da), g["da"], g["mda"], dtype, (72, 136, 8, 44), "da")
    close(host(db), g["db"], g["mdb"], dtype, (72, 136, 8, 44), "db")


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_no_rows_at_all(dtype):
    p = Problem(25, 0, 2, 3, 64, 64, 16, dtype)
    assert p.forward().shape == (0, 64)
    dx, da, db = p.backward(torch.zeros(0, 16, device="cuda"), da=torch.full_like(p.a, 9), db=torch.full_like(p.b, 9))
    assert dx.shape == (0, 64) and not da.any() and not db.any()


@pytest.mark.parametrize("dtype,big", [(F16, 60000.0), (BF16, 2.0 ** 100)])
def test_shrunk_rows_beyond_the_element_type(dtype, big):
    """h is kept in fp32: values of x that drive it beyond binary16's range (or
    far from 1 in bf16), undone by small B, come out right."""
    p = Problem(26, 40, 2, 4, 264, 512, 16, dtype)
    p.x.fill_(0)
    p.x[:, 3] = big
    p.a[:, :, 3] = 8.0
    p.a[:, 5, 3] = 2.0 ** -14
    p.b.mul_(1 / big)
    p.base.zero_()
    h = torch.zeros(p.P, 16, device="cuda")
    ref = p.oracle()
    out = p.forward(h=h)
    assert float(h.abs().max()) == 8 * float(p.x[0, 3])
    close(host(out), ref["out"], ref["mag"], dtype, p.len, "out")
    p.dy.mul_(1 / big)
    g = p.oracle_grad(host(h))
    _, da, db = p.backward(h)
    # dh is kept in fp32: where dy * b falls below its normal range (2^-100 *
    # 2^-100 here in bf16, against 2^-126), each of its N products is off by at
    # most 2^-126, and da = sum_s dh x by N * 2^-126 * sum_s |x|.
    floor = p.N * 2.0 ** -126 * np.abs(host(p.x)).sum()
    close(host(da), g["da"], g["mda"], dtype, p.len, "da", floor)
    close(host(db), g["db"], g["mdb"], dtype, p.len, "db")


def _weight_grads(dtype, off, h, dy, x, a, b, srt=None):
    """dA, dB and the oracle's, for identity rows (or the table srt)."""
    P, R = h.shape
    kw = dict(a_row="sorted", out_row="sorted")
    _, da, db = mq.grouped_lora_backward(dy, x, a, b, h, dev(off), None if srt is None else dev(srt), 1,
                                         need_dx=False, **kw)
    clean = lambda t: np.nan_to_num(host(t), posinf=0, neginf=0)
    return da, db, oracle.grouped_lora_backward(clean(dy), clean(x), host(a), host(b), clean(h), off, srt, 1, **kw)


@pytest.mark.parametrize("spread,run", [(20, 1), (-20, 1), (30, 32), (-30, 32), (7, 32)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gradients_of_low_rank_values_of_very_different_magnitude(dtype, spread, run):
    """h falls (or grows) by 2^spread over the ranks (run 1), or in steps of
    2^spread / 4 over the tiles of `run` rows.  In f16 a value is kept to at
    least 2^-25 2^-10 of the largest of its group in each of its two parts, at
    the split and where its tile is brought to the scale of a larger one:
    floor = 4 * 2^-35 max |h| sum_s |dy[s][n]|."""
    rng = np.random.default_rng(50)
    P, N, K, R = 300, 136, 72, 16
    off = np.array([0, 160, 160, 300], np.int32)
    x, dy = values(rng, (P, K), dtype), values(rng, (P, N), dtype)
    a, b = values(rng, (3, R, K), dtype, 0.1), values(rng, (3, N, R), dtype)
    e = -spread * np.arange(R) / R * np.ones((P, 1)) if run == 1 else -spread / 4 * (np.arange(P) // run)[:, None]
    h = dev((rng.standard_normal((P, R)) * 2.0 ** np.round(e)).astype(np.float32))
    da, db, g = _weight_grads(dtype, off, h, dy, x, a, b)
    floor = np.zeros((3, N, 1))
    if dtype == F16:
        for i in range(3):
            r = slice(off[i], off[i + 1])
            floor[i, :, 0] = 2.0 ** -33 * np.abs(host(h)[r]).max(initial=0) * np.abs(host(dy)[r]).sum(0)
    close(host(db), g["db"], g["mdb"], dtype, (N, K, R, P), "db", floor)
    close(host(da), g["da"], g["mda"], dtype, (N, K, R, P), "da")


@pytest.mark.parametrize("order", [(0, -10, 4, -7, -12), (-12, -7, 0, 4, -10), (4, 0, -7, -10, -12)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gradients_of_columns_that_only_one_tile_of_rows_reaches(dtype, order):
    """h in steps of a power of two over the tiles, and dy's columns nonzero in
    one tile each: every tile's values meet the output alone, whatever scale
    the sums of the others took (floor as above)."""
    rng = np.random.default_rng(54)
    P, N, K, R = 160, 200, 64, 40
    off = np.array([0, P], np.int32)
    x, dy = values(rng, (P, K), dtype), values(rng, (P, N), dtype)
    tile = np.arange(P) // 32
    dy[torch.from_numpy(tile[:, None] != np.arange(N) % 5).cuda()] = 0
    a, b = values(rng, (1, R, K), dtype, 0.1), values(rng, (1, N, R), dtype)
    h = dev((rng.standard_normal((P, R)) * 2.0 ** np.array(order)[tile][:, None]).astype(np.float32))
    _, db, g = _weight_grads(dtype, off, h, dy, x, a, b)
    floor = 2.0 ** -33 * np.abs(host(h)).max() * np.abs(host(dy)).sum(0)[:, None] if dtype == F16 else 0.0
    close(host(db)[0], g["db"][0], g["mdb"][0], dtype, (N, K, R, P), "db", floor)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_infinite_low_rank_values_beside_much_larger_finite_ones(dtype):
    rng = np.random.default_rng(51)
    P, N, K, R = 128, 64, 64, 8
    off = np.array([0, P], np.int32)
    x, dy = values(rng, (P, K), dtype), values(rng, (P, N), dtype).abs() + 1
    a, b = values(rng, (1, R, K), dtype), values(rng, (1, N, R), dtype)
    h = dev((rng.standard_normal((P, R)) * 2.0 ** -60).astype(np.float32))
    h[64:] *= 2.0 ** 60
    h[3, 2] = float("inf")
    _, db, g = _weight_grads(dtype, off, h, dy, x, a, b)
    assert torch.all(db[0, :, 2] == float("inf"))
    keep = np.arange(R) != 2
    floor = 2.0 ** -33 * np.abs(host(h)[64:]).max() * np.abs(host(dy)).sum(0)[:, None] if dtype == F16 else 0.0
    close(host(db)[0][:, keep], g["db"][0][:, keep], g["mdb"][0][:, keep], dtype, (N, K, R, P), "db", floor)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_whole_tiles_of_rows_without_a_pair(dtype):
    """A table whose ids skip rows 32 .. 95 of a group, and a whole group: what
    the skipped rows hold, NaN too, is not read."""
    rng = np.random.default_rng(52)
    P, N, K, R = 200, 72, 136, 24
    off = np.array([0, 130, 200], np.int32)
    srt = np.arange(P, dtype=np.int32)
    srt[32:96] = -1
    srt[130:] = -1
    x, dy = values(rng, (P, K), dtype), values(rng, (P, N), dtype)
    a, b = values(rng, (2, R, K), dtype, 0.1), values(rng, (2, N, R), dtype)
    h = dev(rng.standard_normal((P, R)).astype(np.float32))
    skip = torch.from_numpy(srt < 0).cuda()
    for t in (x, dy, h):
        t[skip] = float("nan")
    da, db, g = _weight_grads(dtype, off, h, dy, x, a, b, srt)
    close(host(da), g["da"], g["mda"], dtype, (N, K, R, P), "da")
    close(host(db), g["db"], g["mdb"], dtype, (N, K, R, P), "db")
    assert not da[1].any() and not db[1].any()


# Both sides of the forward call's choice of one launch or two, at ranks that
# fill no MFMA tile, rows without a group, and groups that end inside a tile.
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,E,N,K,R", [(1, 3, 1032, 8, 8), (17, 2, 1016, 264, 40), (70, 5, 2056, 1024, 64),
                                       (70, 5, 2056, 1032, 64), (300, 40, 3000, 136, 24), (900, 2, 4096, 512, 16)])
def test_forward_of_few_rows(T, E, N, K, R, dtype):
    p = Problem(53, T, 1, E, N, K, R, dtype, out_row="pair", kind="repeat", skip=0.2)
    ref = p.oracle()
    h = torch.full((p.P, R), 3.0, device="cuda")
    out = p.forward(out=torch.full((p.P, N), 7.0, dtype=dtype, device="cuda"), h=h)
    close(host(out), ref["out"], ref["mag"], dtype, p.len, "out")
    assert np.array_equal(host(out)[~ref["written"]], host(p.base)[~ref["written"]])
    xh = np.abs(host(p.x))[np.maximum(p.srt[:p.n], 0)]
    mh = np.concatenate([xh[p.off[e]:p.off[e + 1]] @ np.abs(host(p.a[e])).T for e in range(E)])
    close(host(h)[:p.n], ref["h"][:p.n], mh, F32, p.len, "h")
    assert np.all(host(h)[p.n:] == 3)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_infinities_and_nans_stay_in_their_rows_and_groups(dtype):
    p = Problem(27, 60, 2, 4, 136, 264, 16, dtype)
    out0, h = p.forward(), torch.zeros(p.P, 16, device="cuda")
    p.forward(h=h)
    dx0, da0, db0 = p.backward(h)
    s = int(p.off[1]) + 1                      # a row of group 1
    t = int(p.srt[s]) // 2
    p.x[t, 7] = float("inf")
    out1 = p.forward()
    rows = torch.from_numpy(p.srt // 2 == t).cuda()
    assert torch.equal(out0[~rows], out1[~rows]) and not torch.isfinite(out1[rows]).any()
    p.x[t, 7] = 0
    p.dy[s, 3] = float("nan")
    dx1, da1, db1 = p.backward(h)
    keep = torch.arange(p.P, device="cuda") != s
    assert torch.equal(dx0[keep], dx1[keep]) and torch.isnan(dx1[s]).all()
    for e in (0, 2, 3):
        assert torch.equal(db0[e], db1[e])
    assert torch.isnan(da1[1]).all() and torch.isnan(db1[1, 3]).all()
    assert torch.isfinite(db1[1, :3]).all() and torch.isfinite(db1[1, 4:]).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gradients_against_differences_of_the_forward_call(dtype):
    """out is linear in each of x, a and b: with base = 0 and weights g on out,
    <g, f(v + d) - f(v - d)> / 2 = <gradient, d>.  v +- d is exact (v, d on a
    coarse grid); f rounds each output by half a step, which the left side sums
    over T*k*N outputs with random signs (4 sqrt(count) of them)."""
    T, k, E, N, K, R = 64, 2, 4, 136, 136, 16
    p = Problem(28, T, k, E, N, K, R, dtype, kind="repeat", skip=0.1)
    rng = np.random.default_rng(29)
    grid = lambda t: t.copy_((t.float() * 8).round() / 8)
    for t in (p.x, p.a, p.b):
        grid(t)
    g = values(rng, (p.P, N), dtype)
    p.dy[:p.n] = g[:p.n]
    p.dy[p.n:] = 0
    h = torch.zeros(p.P, R, device="cuda")
    p.forward(base=None, h=h)
    dx, da, db = p.backward(h, dx=torch.zeros(p.P, K, dtype=dtype, device="cuda"))
    dxt = mq.moe_permute_backward(dx, p.dp2s, k, out_dtype=F32)
    u = torch.finfo(dtype).eps / 2
    for t, grad in ((p.x, dxt), (p.a, da), (p.b, db)):
        d = grid(values(rng, t.shape, dtype))
        v = t.clone()
        f = []
        for sign in (1, -1):
            t.copy_(v + sign * d)
            f.append(p.forward(base=None, out=torch.zeros(p.P, N, dtype=dtype, device="cuda")).double())
        t.copy_(v)
        lhs = float((p.dy.double() * (f[0] - f[1])).sum()) / 2
        rhs = float((grad.double() * d.double()).sum())
        noise = u * float(((p.dy.double() * f[0]).square() + (p.dy.double() * f[1]).square()).sum().sqrt())
        noise += u * float((grad.double() * d.double()).square().sum().sqrt()) * (k ** 0.5)
        assert abs(lhs - rhs) <= 4 * noise, (lhs, rhs, noise)


def test_offsets_past_32_bits():
    """More than 2^31 elements of output rows (4.4 GB of bf16)."""
    T, N, K, R = 2 ** 16 + 100, 32776, 64, 8
    rng = np.random.default_rng(30)
    ids = rng.integers(0, 3, (T, 1)).astype(np.int32)
    off, srt, p2s, _ = oracle.route_prep(ids, 3)
    x, a, b = values(rng, (T, K), BF16), values(rng, (3, R, K), BF16, 0.1), values(rng, (3, N, R), BF16)
    h = torch.zeros(T, R, device="cuda")
    out = mq.grouped_lora(x, a, b, dev(off), dev(srt), 1, out_row="pair", pair_to_sorted=dev(p2s), h=h)
    assert out.numel() > 2 ** 31
    for t in (0, 1, T // 3, T - 2, T - 1):
        e = int(ids[t, 0])
        ref = host(b[e]) @ (host(a[e]) @ host(x[t]))
        mag = np.abs(host(b[e])) @ (np.abs(host(a[e])) @ np.abs(host(x[t])))
        close(host(out[t]), ref, mag, BF16, (K, N, R, 1), t)
    dx, da, db = mq.grouped_lora_backward(out, x, a, b, h, dev(off), dev(srt), 1, out_row="pair")
    s = T - 1
    t, e = int(srt[s]), 2
    ref = host(a[e]).T @ (host(b[e]).T @ host(out[t]))
    mag = np.abs(host(a[e])).T @ (np.abs(host(b[e])).T @ np.abs(host(out[t])))
    close(host(dx[s]), ref, mag, BF16, (K, N, R, 1), "dx")
    i = srt[off[2]:off[3]]
    cols = slice(N - 16, N)
    o, hh = host(out[torch.from_numpy(i).long().cuda()][:, cols]), host(h)[off[2]:off[3]]
    close(host(db[2, cols]), o.T @ hh, np.abs(o).T @ np.abs(hh), BF16, (K, N, R, T), "db")


def _layer(p, d, route, q, bufs):
    """One training step of adapters beside a frozen NVFP4 down projection:
    route -> FC1 -> FC2 + adapters (in place) -> combine, and back to the
    adapters, the routing weights and FC1's output."""
    ids, tw, dout = q["ids"], q["tw"], q["dout"]
    E, k = d["E"], d["k"]
    off, srt, p2s, _ = mq.moe_route_prep(ids, E, out=route, workspace=bufs["rws"])
    mq.grouped_gemm_qnvfp4(q["x"], q["w1"], q["s1"], q["g1"], off, srt, k, act="silu_mul", out=bufs["h1"])
    mq.grouped_gemm_qnvfp4(bufs["h1"], q["w2"], q["s2"], q["g2"], off, srt, k, a_row="sorted", out=bufs["y"])
    mq.grouped_lora(bufs["h1"], q["a"], q["b"], off, srt, k, base=bufs["y"], scale=q["scale"], a_row="sorted",
                    out=bufs["y"], h=bufs["h"], workspace=bufs["ws"])
    mq.moe_scatter_combine(bufs["y"], p2s, tw, out=bufs["out"])
    mq.moe_scatter_combine_backward(dout, bufs["y"], p2s, tw, dy=bufs["dy"], dw=bufs["dw"])
    mq.grouped_lora_backward(bufs["dy"], bufs["h1"], q["a"], q["b"], bufs["h"], off, srt, k, scale=q["scale"],
                             a_row="sorted", dx=bufs["dx"], da=bufs["da"], db=bufs["db"], workspace=bufs["wsb"])
    mq.moe_permute(q["x"], p2s, k, out=bufs["xs"])
    mq.moe_permute_backward(bufs["xs"], p2s, k, out=bufs["xt"])


def _layer_problem(T=96, E=12, k=3, H=512, I=256, R=16, dtype=BF16):
    d = synth.nvfp4_moe(41, T, E, k, H, I, routing="zipf" if E > 40 else "repeat")
    rng = np.random.default_rng(42)
    q = dict(ids=dev(d["topk_ids"]), tw=dev(d["topk_weights"]), x=dev(d["x"]), w1=dev(d["w1"]), s1=dev(d["s1"]),
             g1=dev(d["g1"]), w2=dev(d["w2"]), s2=dev(d["s2"]), g2=dev(d["g2"]), a=values(rng, (E, R, I), dtype, I ** -0.5),
             b=values(rng, (E, H, R), dtype, R ** -0.5), scale=dev(rng.random(E).astype(np.float32) + 0.5),
             dout=values(rng, (T, H), dtype, 0.1))
    P = T * k
    i32 = dict(dtype=torch.int32, device="cuda")
    z = lambda *s, dt=dtype: torch.zeros(*s, dtype=dt, device="cuda")
    route = (torch.empty(E + 1, **i32), torch.empty(P, **i32), torch.empty(P, **i32), torch.empty(1, **i32))
    bufs = dict(rws=z(max(1, mq.route_workspace_bytes(T, k, E)), dt=torch.uint8), h1=z(P, I), y=z(P, H),
                h=z(P, R, dt=F32), out=z(T, H), dy=z(P, H), dw=z(T, k, dt=F32), dx=z(P, I), da=z(E, R, I),
                db=z(E, H, R), xs=z(P, H), xt=z(T, H), ws=z(mq.lora_workspace_bytes(P, E, H, I, R), dt=torch.uint8),
                wsb=z(mq.lora_workspace_bytes(P, E, H, I, R, backward=True), dt=torch.uint8))
    return d, q, route, bufs


def test_training_step_of_adapters_beside_the_quantized_layer():
    """Every step checked from the stored input of that step (the tensors the
    next call reads), so that no tolerance spans two roundings."""
    d, q, route, bufs = _layer_problem()
    _layer(None, d, route, q, bufs)
    k, off, srt, p2s = d["k"], *(host(t) for t in route[:3])
    h1, sc = host(bufs["h1"]), host(q["scale"])
    y0 = mq.grouped_gemm_qnvfp4(bufs["h1"], q["w2"], q["s2"], q["g2"], route[0], route[1], k, a_row="sorted")
    n, dims = int(off[-1]), (256, 512, 16, p2s.size)
    f = oracle.grouped_lora(h1, host(q["a"]), host(q["b"]), off, srt, k, base=host(y0), scale=sc, a_row="sorted")
    close(host(bufs["y"])[:n], f["out"][:n], f["mag"][:n], BF16, dims, "y")
    y, w = host(bufs["y"]), host(q["tw"])
    ref = oracle.scatter_combine(y, p2s, w)
    assert np.all(np.abs(host(bufs["out"]) - ref) <= half_step(ref, BF16) +
                  2 * k * 2.0 ** -24 * oracle.scatter_combine(np.abs(y), p2s, w))
    dy, dw = oracle.scatter_combine_backward(host(q["dout"]), y, p2s, w)
    _, mdw = oracle.scatter_combine_backward(np.abs(host(q["dout"])), np.abs(y), p2s, w)
    assert np.all(np.abs(host(bufs["dy"]) - dy) <= half_step(dy, BF16) + 2.0 ** -24 * np.abs(dy))
    assert np.all(np.abs(host(bufs["dw"]) - dw) <= 32 * 2.0 ** -24 * mdw)
    g = oracle.grouped_lora_backward(host(bufs["dy"]), h1, host(q["a"]), host(q["b"]), host(bufs["h"]), off, srt, k,
                                     scale=sc, a_row="sorted")
    close(host(bufs["dx"])[:n], g["dx"][:n], g["mdx"][:n], BF16, dims, "dx")
    close(host(bufs["da"]), g["da"], g["mda"], BF16, dims, "da")
    close(host(bufs["db"]), g["db"], g["mdb"], BF16, dims, "db")


def test_training_step_captured_and_replayed():
    from tests.test_gpu_graphs import _capture_and_replay
    d, q, route, bufs = _layer_problem(T=1100, E=48, k=2)
    outputs = [bufs[n] for n in ("y", "h", "out", "dy", "dw", "dx", "da", "db", "xs", "xt")]
    _capture_and_replay(lambda: _layer(None, d, route, q, bufs), outputs)


def test_serving_step_captured_and_replayed():
    # a batch of single tokens, adapters by request, out of place in the batch's order
    from tests.test_gpu_graphs import _capture_and_replay
    p = Problem(43, 19, 1, 8, 520, 1032, 16, F16, out_row="pair", kind="repeat", skip=0.3)
    out = torch.zeros(p.P, p.N, dtype=F16, device="cuda")
    ws = torch.zeros(mq.lora_workspace_bytes(p.P, p.E, p.N, p.K, p.R), dtype=torch.uint8, device="cuda")
    _capture_and_replay(lambda: p.forward(out=out, workspace=ws), [out])


def test_two_streams_at_once_with_their_own_workspaces():
    p = Problem(44, 600, 2, 6, 1032, 520, 32, BF16)
    h = torch.zeros(p.P, p.R, device="cuda")
    out = p.forward(h=h)
    ref = p.backward(h)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append((p.forward(), *p.backward(h)))
        torch.cuda.synchronize()
        for g in got:
            for v, r in zip(g, (out, *ref)):
                assert torch.equal(v, r)


def test_tables_with_ids_out_of_range_skip_those_rows():
    """A table that route prep never writes: ids outside [0, P) skip their
    rows in every call, and nothing out of range is touched."""
    p = Problem(45, 40, 2, 4, 136, 264, 16, BF16)
    srt = p.srt.copy()
    srt[5], srt[17] = -1, p.P
    h = torch.full((p.P, 16), 3.0, device="cuda")
    out = torch.full((p.P, 136), 7.0, dtype=BF16, device="cuda")
    p.dsrt = dev(srt)
    p.forward(out=out, h=h)
    full = oracle.grouped_lora(host(p.x), host(p.a), host(p.b), p.off, p.srt, 2, base=host(p.base), scale=p.scale)
    keep = np.ones(p.P, bool)
    keep[[5, 17]] = False
    close(host(out)[keep], full["out"][keep], full["mag"][keep], BF16, p.len, "out")
    assert np.all(host(out)[~keep] == 7)
    hh = host(h)
    hh[~keep] = 0
    g = p.oracle_grad(hh)
    dyz = host(p.dy)
    dyz[~keep] = 0
    g = oracle.grouped_lora_backward(dyz, host(p.x), host(p.a), host(p.b), hh, p.off, p.srt, 2, scale=p.scale)
    h[torch.from_numpy(~keep).cuda()] = float("nan")
    dx = torch.full((p.P, 264), 7.0, dtype=BF16, device="cuda")
    _, da, db = p.backward(h, dx=dx)
    close(host(dx)[keep], g["dx"][keep], g["mdx"][keep], BF16, p.len, "dx")
    assert np.all(host(dx)[~keep] == 7)
    close(host(da), g["da"], g["mda"], BF16, p.len, "da")
    close(host(db), g["db"], g["mdb"], BF16, p.len, "db")


def test_offsets_that_reach_past_the_rows_are_clamped():
    p = Problem(46, 16, 2, 3, 72, 72, 8, F16)
    off = p.off.copy()
    off[-1] = p.P + 1000
    p.doff = dev(off)
    ref = p.oracle()
    out = p.forward(pair_to_sorted=None)
    close(host(out), ref["out"], ref["mag"], F16, p.len, "out")


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_very_long_groups_of_short_rows(dtype):
    """Hundreds of chunks a group, joined in order; a group between them and
    the last one without rows."""
    rng = np.random.default_rng(56)
    P, N, K, R = 700_000, 16, 8, 8
    off = np.array([0, 250_001, 250_001, 699_990, 699_990], np.int32)
    x, dy = values(rng, (P, K), dtype), values(rng, (P, N), dtype, 0.1)
    a, b = values(rng, (4, R, K), dtype, 0.3), values(rng, (4, N, R), dtype, 0.3)
    h = torch.zeros(P, R, device="cuda")
    out = torch.full((P, N), 7.0, dtype=dtype, device="cuda")
    mq.grouped_lora(x, a, b, dev(off), None, 1, a_row="sorted", out=out, h=h)
    ref = oracle.grouped_lora(host(x), host(a), host(b), off, None, 1, a_row="sorted", P=P)
    n = int(off[-1])
    close(host(out)[:n], ref["out"][:n], ref["mag"][:n], dtype, (K, N, R), "out")
    assert np.all(host(out)[n:] == 7)
    dx, da, db = mq.grouped_lora_backward(dy, x, a, b, h, dev(off), None, 1, a_row="sorted",
                                          dx=torch.full((P, K), 7.0, dtype=dtype, device="cuda"))
    g = oracle.grouped_lora_backward(host(dy), host(x), host(a), host(b), host(h), off, None, 1, a_row="sorted")
    close(host(dx)[:n], g["dx"][:n], g["mdx"][:n], dtype, (K, N, R), "dx")
    assert np.all(host(dx)[n:] == 7)
    close(host(da), g["da"], g["mda"], dtype, (K, N, R, P), "da")
    close(host(db), g["db"], g["mdb"], dtype, (K, N, R, P), "db")


def test_two_launch_forward_captured_and_replayed():
    from tests.test_gpu_graphs import _capture_and_replay
    p = Problem(57, 300, 2, 8, 1032, 5000, 40, BF16, out_row="pair", kind="repeat", skip=0.2)
    out, h = torch.zeros(p.P, p.N, dtype=BF16, device="cuda"), torch.zeros(p.P, p.R, device="cuda")
    need = mq.lora_workspace_bytes(p.P, p.E, p.N, p.K, p.R)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    # (rows of h without a group are not written)
    _capture_and_replay(lambda: p.forward(out=out, h=h, workspace=ws), [out, h[:p.n]])
