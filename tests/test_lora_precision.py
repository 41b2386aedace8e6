"""What the adapters keep of the fp32 low-rank values (h, dh) on their way
through 16-bit MFMA parts, apart from the sums around them.

A value enters as three bf16 parts, exactly, or as two binary16 parts, to
2^-23 of itself plus an absolute floor: 2^-33 of its row's largest value in the
forward call and dx, 2^-35 of its 32-row tile's (and so of its group's) in da
and db."""
import numpy as np
import pytest
import torch

from tests.gpu_util import dev, host
from tests.test_gpu_permute import BF16, F16, half_step

mq = pytest.importorskip("quantized_moe_grouped_route_amd")


@pytest.fixture(scope="module")
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mq.lib()


def within(got, ref, tol, dtype):
    over = np.isinf(got) & (np.sign(got) == np.sign(ref)) & (np.abs(ref) + tol >= torch.finfo(dtype).max)
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - ref) <= tol) & ~over
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], ref[bad][:3], tol[bad][:3])


# Exponents of the 32-row tiles of one group: a large tile before smaller ones,
# after them, between them; steps; and more than 2^80 apart, where small tiles
# are dropped.
SPREADS = [(0, *[-45] * 12), (0, *[-60] * 12), (*[-60] * 12, 0), (-60, -60, 0, -60, -60, -60),
           (0, -30, -60, -34, -38, -42, -46, -50), (0, -60, 20, -60), (0, -78, -70, -78), (0, -90, -100, -90)]


@pytest.mark.gpu
@pytest.mark.parametrize("exps", SPREADS, ids=["_".join(map(str, e[:4])) + f"x{len(e)}" for e in SPREADS])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_db_of_tiles_far_below_their_groups_largest_value(gpu, dtype, exps):
    """h of one sign in tiles of 32 rows times 2^exps; dy zero for the largest
    tile, elsewhere nonzero in the tile's own columns and in columns that all
    the small ones share, so that only they reach db.

    tol = half step + per value 2^-23 (f16's parts) + 2^-24 for each addition of
    the P rows' 3 parts, independent, 4 sqrt(3 P) of them + in f16 the tile's
    floor for each of its rows, 2^-35 of its largest value, or 2^-80 of the
    group's for a dropped tile + P values of fp32 below its normal range."""
    rng = np.random.default_rng(61)
    tiles, R, N, K = len(exps), 24, 72, 16
    P = 32 * tiles
    # the smallest at 2^0 .. 2^3, the largest at 2^(4 m + 2), which f16's tile
    # scale brings to the lowest place that it allows
    e = np.array(exps) - min(exps)
    e += (2 - max(e)) % 4
    e = np.repeat(e, 32).astype(np.float64)
    h = ((1 + rng.random((P, R))) * 2.0 ** e[:, None]).astype(np.float32)
    tile = np.arange(P) // 32
    dy = 1 + rng.integers(0, 4, (P, N)).astype(np.float32)
    dy[(tile[:, None] != np.arange(N) % (tiles + 1)) & (np.arange(N) % (tiles + 1) != tiles)] = 0
    dy[e == e.max()] = 0
    x = torch.zeros(P, K, dtype=dtype).cuda()
    a, b = torch.zeros(1, R, K, dtype=dtype).cuda(), torch.zeros(1, N, R, dtype=dtype).cuda()
    _, _, db = mq.grouped_lora_backward(dev(dy).to(dtype), x, a, b, dev(h), dev(np.array([0, P], np.int32)), None, 1,
                                        a_row="sorted", need_dx=False)
    h, dy = h.astype(np.float64), dy.astype(np.float64)
    ref = dy.T @ h
    tol = half_step(ref, dtype) + (2.0 ** -23 + 4 * np.sqrt(3 * P) * 2.0 ** -24) * ref + P * 2.0 ** -126
    if dtype == F16:
        top = np.repeat(h.reshape(tiles, -1).max(1), 32)
        floor = np.where(e < e.max() - 80, 2.0 ** -80 * h.max(), 2.0 ** -35 * top)
        tol += (dy * floor[:, None]).sum(0)[:, None]
    within(host(db)[0], ref, tol, dtype)


# ------------------------------------------- every bit of the low-rank values
# h (dh) are made of integers v as wide as the parts carry, 24 bits in bf16 and
# 23 in f16, in neighbours v and v + 1 that the second product subtracts: the
# leading parts cancel, and what is left are integers of at most 16 times a power
# of two.  Every fp32 value on the way is exact (only one 32-wide step of the
# contraction meets a column, and its parts add from the largest down), so the
# outputs have to be equal; a lost part leaves about half of them wrong.
BITS = {F16: 23, BF16: 24}


def neighbours(rng, shape, dtype):
    """Integers of shape [..., even]: v, v + 1, v', v' + 1, ..."""
    top = 2 ** (BITS[dtype] - 1)
    v = rng.integers(top, 2 * top - 2, (*shape[:-1], shape[-1] // 2))
    return np.stack([v, v + 1], -1).reshape(shape)


def digits(v):
    """v = sum_j digits[j] * 2^(16, 8, 0), each exact in 8 bits."""
    return np.stack([v >> 16, v >> 8 & 255, v & 255], -1).astype(np.float32)


WEIGHTS = np.array([256, 1, 1 / 256], np.float32)   # times the digits: v / 2^8


def signs(rng, n, length):
    """[n][length]: +-1 on the second of each pair, the opposite on the first, in
    one 32-wide step for each row, zero in the others."""
    s = rng.choice([-1, 1], (n, (length + 1) // 2))
    full = np.stack([-s, s], -1).reshape(n, -1)[:, :length]
    if length % 2:
        full[:, -1] = 0
    steps = max(1, (length + 31) // 32)
    return np.where(np.arange(length) // 32 == np.arange(n)[:, None] % steps, full, 0).astype(np.float32)


def kept(v, dtype, parts):
    """The sum of the first parts of v."""
    v = torch.from_numpy(np.asarray(v, np.float32)).clone()
    out = torch.zeros_like(v)
    for _ in range(parts):
        p = (v * 2.0 ** -14).to(dtype).float() * 2.0 ** 14 if dtype == F16 else v.to(dtype).float()
        out, v = out + p, v - p
    return out.double().numpy()


@pytest.mark.parametrize("R", [8, 64, 256])
@pytest.mark.parametrize("dtype,parts", [(F16, 2), (BF16, 3)])
def test_the_integers_need_every_part(dtype, parts, R):
    rng = np.random.default_rng(62)
    v, s = neighbours(rng, (R,), dtype), signs(rng, 72, R).astype(np.float64)
    assert np.array_equal(digits(v) @ WEIGHTS, v / 256)
    assert np.array_equal(s @ kept(v, dtype, parts), s @ v)
    assert np.abs(s @ v).max() <= 16
    assert np.mean(s @ kept(v, dtype, parts - 1) != s @ v) > 0.4


# One launch for ranks of one, two and four MFMA tiles; two launches with the
# weights of 32 and 64 ranks in registers, and reloaded for more.
SHAPES = [  # P, E, N, K, R
    (40, 3, 136, 64, 8), (40, 3, 136, 264, 32), (40, 3, 136, 264, 64), (40, 3, 1032, 8200, 16), (300, 4, 392, 8192, 32),
    (90, 5, 136, 2056, 64), (90, 5, 136, 64, 72), (90, 2, 392, 136, 128), (70, 3, 136, 72, 256),
]


def groups(rng, P, E):
    """Offsets of E groups, one of them empty, that leave 3 rows without one."""
    cut = np.sort(rng.integers(0, P - 2, E - 1))
    if E > 2:
        cut[1] = cut[0]
    return np.concatenate([[0], cut, [P - 3]]).astype(np.int32)


def rank_side(rng, dtype, off, P, E, wide, R):
    """A weight [E][R][wide] and rows [P][wide] whose products are v[e][r] * 2^(e_s
    - 8), and those."""
    v = neighbours(rng, (E, R), dtype)
    at = [0, wide // 2, wide - 1]
    w, rows = np.zeros((E, R, wide), np.float32), np.zeros((P, wide), np.float32)
    es = rng.integers(-3, 4, P)
    w[:, :, at] = digits(v)
    rows[:, at] = WEIGHTS * 2.0 ** es[:, None]
    e = np.searchsorted(off, np.arange(P), side="right") - 1
    low = np.where((np.arange(P) < off[-1])[:, None], v[np.minimum(e, E - 1)] * 2.0 ** (es[:, None] - 8), 0.0)
    return w, rows, low, np.minimum(e, E - 1)


@pytest.mark.gpu
@pytest.mark.parametrize("P,E,N,K,R", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_out_is_exact_where_the_low_rank_values_cancel(gpu, dtype, P, E, N, K, R):
    rng = np.random.default_rng(63)
    off = groups(rng, P, E)
    a, x, low, e = rank_side(rng, dtype, off, P, E, K, R)
    b = np.stack([signs(rng, N, R) for _ in range(E)])
    sc = np.array([0.5, -2, 1, 4, -0.25], np.float32)[:E]
    h = torch.zeros(P, R, device="cuda")
    out = torch.zeros(P, N, dtype=dtype, device="cuda")
    mq.grouped_lora(dev(x).to(dtype), dev(a).to(dtype), dev(b).to(dtype), dev(off), None, 1, a_row="sorted",
                    scale=dev(sc), out=out, h=h)
    assert np.array_equal(host(h), low)
    ref = np.stack([sc[e[s]] * (b[e[s]].astype(np.float64) @ low[s]) for s in range(P)])
    assert np.abs(ref).max() > 0
    assert np.array_equal(host(out), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("P,E,N,K,R", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_dx_is_exact_where_the_low_rank_values_cancel(gpu, dtype, P, E, N, K, R):
    rng = np.random.default_rng(64)
    off = groups(rng, P, E)
    bt, dy, low, e = rank_side(rng, dtype, off, P, E, N, R)
    a = np.stack([signs(rng, K, R).T for _ in range(E)])
    sc = np.array([0.5, -2, 1, 4, -0.25], np.float32)[:E]
    dx = torch.zeros(P, K, dtype=dtype, device="cuda")
    mq.grouped_lora_backward(dev(dy).to(dtype), torch.zeros(P, K, dtype=dtype).cuda(), dev(a).to(dtype),
                             dev(bt.transpose(0, 2, 1)).to(dtype), torch.zeros(P, R).cuda(), dev(off), None, 1,
                             a_row="sorted", scale=dev(sc), dx=dx)
    ref = np.stack([sc[e[s]] * (low[s] @ a[e[s]].astype(np.float64)) for s in range(P)])
    assert np.abs(ref).max() > 0
    assert np.array_equal(host(dx), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("P,E,N,K,R", [*SHAPES, (2500, 2, 136, 72, 40)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_weight_gradients_are_exact_where_the_low_rank_values_cancel(gpu, dtype, P, E, N, K, R):
    """The contraction runs over a group's rows, 32 in a step: h and dh hold
    v[s] * 2^(r % 4 - 8), and dy and x subtract neighbouring rows."""
    rng = np.random.default_rng(65)
    off = groups(rng, P, E)
    v = np.zeros(P, np.int64)
    x, dys = np.zeros((P, K), np.float32), np.zeros((P, N), np.float32)
    for g in range(E):
        r, n = slice(off[g], off[g + 1]), int(off[g + 1] - off[g])
        v[r] = neighbours(rng, (n + n % 2,), dtype)[:n]
        x[r], dys[r] = signs(rng, K, n).T, signs(rng, N, n).T
    col = (2.0 ** (np.arange(R) % 4)).astype(np.float32)
    low = v[:, None] / 256 * col.astype(np.float64)
    sc = np.array([0.5, -2, 1, 4, -0.25], np.float32)[:E]
    zero = lambda *s: torch.zeros(*s, dtype=dtype).cuda()
    doff, kw = dev(off), dict(a_row="sorted", scale=dev(sc), need_dx=False)
    ref = lambda wide: np.stack([sc[g] * (low[off[g]:off[g + 1]].T @ wide[off[g]:off[g + 1]].astype(np.float64))
                                 for g in range(E)])
    _, _, db = mq.grouped_lora_backward(dev(dys).to(dtype), zero(P, K), zero(E, R, K), zero(E, N, R),
                                        dev(low.astype(np.float32)), doff, None, 1, **kw)
    want = ref(dys).transpose(0, 2, 1)
    assert np.abs(want).max() > 0
    assert np.array_equal(host(db), want)
    at = [0, N // 2, N - 1]
    dy, b = np.zeros((P, N), np.float32), np.zeros((E, N, R), np.float32)
    dy[:, at], b[:, at, :] = digits(v), WEIGHTS[:, None] * col
    _, da, _ = mq.grouped_lora_backward(dev(dy).to(dtype), dev(x).to(dtype), zero(E, R, K), dev(b).to(dtype),
                                        torch.zeros(P, R).cuda(), doff, None, 1, **kw)
    assert np.array_equal(host(da), ref(x))


# ----------------------------------------- low-rank values of very different size
def spread_values(rng, dtype, E, R, wide, spread):
    """Weight [E][R][wide] and the three columns that it uses: rank r near
    2^(-spread * r / R), from two factors where one type's range ends."""
    w = np.zeros((E, R, wide), np.float32)
    ex = -np.round(spread * np.arange(R) / R)
    w[:, ex > -14, 0] = ((1 + rng.random((E, R))) * 2.0 ** ex)[:, ex > -14]
    mid, low = (ex <= -14) & (ex > -28), ex <= -28
    w[:, mid, wide // 2] = ((1 + rng.random((E, R))) * 2.0 ** (ex + 14))[:, mid]
    w[:, low, wide - 1] = ((1 + rng.random((E, R))) * 2.0 ** (ex + 28))[:, low]
    return torch.from_numpy(w).to(dtype).cuda(), [0, wide // 2, wide - 1]


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [0, 12, 20, 30, 40])
@pytest.mark.parametrize("P,E,N,K,R", [(40, 3, 264, 64, 8), (40, 3, 264, 264, 64), (40, 3, 264, 8200, 16),
                                       (90, 2, 264, 136, 128)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_each_rank_alone_in_a_column(gpu, dtype, P, E, N, K, R, spread):
    """h (dh) falls by 2^spread over the ranks, and every column of out (dx) has
    one rank: nothing hides what that rank lost.  h and dh are single products
    of two 16-bit values, exact in fp32.

    tol = half step + relative 2^-23 (f16's parts) + 4 * 2^-24 (the scale, three
    parts) + in f16 2^-33 of the row's largest scaled value times the weight."""
    rng = np.random.default_rng(66)
    off = groups(rng, P, E)
    n = int(off[-1])
    e = np.searchsorted(off, np.arange(n), side="right") - 1
    sc = (0.5 + rng.random(E)).astype(np.float32)

    def one(weight_wide, other_wide):
        w, at = spread_values(rng, dtype, E, R, weight_wide, spread)
        rows = torch.zeros(P, weight_wide, dtype=dtype)
        rows[:, at] = torch.from_numpy(((1 + rng.random((P, 1))) * np.array([1, 2.0 ** -14, 2.0 ** -28]) * 2.0 ** 14)
                                       .astype(np.float32)).to(dtype)
        # the other weight: column c has rank c % R alone, small for the largest
        # ranks, so that no output leaves f16's range
        rank = np.arange(other_wide) % R
        size = 2.0 ** (np.round(spread * rank / R) / 2 - 10)
        other = np.zeros((E, other_wide, R), np.float32)
        other[:, np.arange(other_wide), rank] = (1 + rng.random((E, other_wide))) * size
        return w, rows.cuda(), torch.from_numpy(other).to(dtype).cuda()

    def check(got, low, other, what):
        s = sc.astype(np.float64)[e][:, None]
        oh, lh = host(other), s * low[:n]
        ref = np.stack([oh[e[i]] @ lh[i] for i in range(n)])
        tol = half_step(ref, dtype) + (2.0 ** -23 + 4 * 2.0 ** -24) * np.abs(ref)
        if dtype == F16:
            tol += 2.0 ** -33 * np.abs(lh).max(1)[:, None] * np.abs(oh).sum(2)[e]
        within(host(got)[:n], ref, tol, dtype)

    doff, dsc = dev(off), dev(sc)
    a, x, b = one(K, N)
    h = torch.zeros(P, R, device="cuda")
    out = mq.grouped_lora(x, a, b, doff, None, 1, a_row="sorted", scale=dsc, h=h)
    check(out, host(h), b, "out")
    bt, dy, at = one(N, K)
    b, a = bt.transpose(1, 2).contiguous(), at.transpose(1, 2).contiguous()
    dx, _, _ = mq.grouped_lora_backward(dy, torch.zeros_like(x), a, b, h, doff, None, 1, a_row="sorted", scale=dsc)
    dh = np.zeros((P, R))
    dh[:n] = np.stack([host(bt)[e[i]] @ host(dy)[i] for i in range(n)])
    check(dx, dh, at, "dx")
