"""moe_permute, its gradient and the gradients of the weighted combine against
the float64 oracle, at the sizes and tables where they can go wrong.

Tolerances, per element: the output's one rounding, half a step
(finfo.eps / 2 relative, plus half the smallest subnormal), and one fp32
rounding (2^-24) of at most the sum of the magnitudes for each addition in a
chain: topk additions for the unweighted sum; for dw's sums over N columns, at
most N / 256 in a thread (8 columns of every 2048, at the least 8), and 16 for
the tree over 256 threads."""
import numpy as np
import pytest
import torch

import oracle
import synth
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

mq = pytest.importorskip("quantized_moe_grouped_route_amd")

F16, BF16, F32, U8 = torch.float16, torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mq.lib()


def half_step(ref, dtype):
    fi = torch.finfo(dtype)
    return np.abs(ref) * fi.eps / 2 + fi.tiny * fi.eps / 2


def tables(seed, T, k, E, kind="distinct", skip=0.0):
    rng = np.random.default_rng(seed)
    if kind == "none":
        ids = np.full((T, k), -1, np.int32)
    elif kind == "one":                         # every slot to the same expert, repeats in a token
        ids = np.full((T, k), E // 2, np.int32)
    elif kind == "repeat":
        ids = synth.uniform_ids_with_repeats(rng, T, k, E)
    else:
        ids = synth.distinct_uniform_ids(rng, T, k, E)
    ids = np.where(rng.random((T, k)) < skip, -1, ids).astype(np.int32)
    return rng, ids, oracle.route_prep(ids, E)


def values(rng, shape, dtype, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(dtype).cuda()


CASES = [  # T, k, E, N, kind, skip
    (0, 2, 4, 64, "distinct", 0.0),
    (1, 1, 1, 8, "distinct", 0.0),
    (1, 8, 256, 7168, "distinct", 0.0),
    (3, 64, 64, 40, "distinct", 0.3),
    (37, 3, 5, 1000, "repeat", 0.3),
    (64, 2, 4, 256, "none", 0.0),
    (130, 4, 7, 2056, "one", 0.0),
    (255, 8, 16, 1032, "repeat", 0.1),         # around one workgroup of tokens per compute unit,
    (257, 8, 16, 1032, "repeat", 0.1),         # where all slots of a token move to one
    (511, 5, 16, 2048, "distinct", 0.1),       # and around two
    (513, 5, 16, 2048, "distinct", 0.1),
    (1023, 2, 8, 4096, "distinct", 0.0),
    (1025, 3, 37, 512, "repeat", 0.2),
    (9, 2, 4, 20000, "distinct", 0.1),
]


@pytest.mark.parametrize("dtype", [F16, BF16, F32, U8])
@pytest.mark.parametrize("T,k,E,N,kind,skip", CASES)
def test_permute_is_the_exact_copy(T, k, E, N, kind, skip, dtype):
    rng, _, (off, srt, p2s, _) = tables(1, T, k, E, kind, skip)
    N = (N + 15) // 16 * 16 if dtype == U8 else N
    x = torch.from_numpy(rng.integers(0, 256, (T, N), dtype=np.uint8)).cuda() if dtype == U8 \
        else values(rng, (T, N), dtype)
    out = torch.full((T * k, N), 7, dtype=dtype, device="cuda")
    got = mq.moe_permute(x, dev(p2s), k, out=out)
    assert got is out
    ref, written = oracle.permute(host(x), p2s, k)
    assert np.array_equal(host(out), np.where(written[:, None], ref, 7))


def test_permute_copies_bits_of_nan_and_infinity():
    x = torch.tensor([[0x7F80, 0xFF80, 0x7F81, 0xFFFF, 0x0001, 0x8000, 0x7FC1, 0x3F80]] * 5, dtype=torch.int32)
    x = x.to(torch.int16).view(BF16).cuda()
    out = mq.moe_permute(x, torch.arange(9, -1, -1, dtype=torch.int32).cuda(), 2)
    assert torch.equal(out.view(torch.int16), x.view(torch.int16).repeat_interleave(2, 0).flip(0))


@pytest.mark.parametrize("dtype,out_dtype", [(F16, F16), (BF16, BF16), (F32, F32), (BF16, F32), (F32, F16)])
@pytest.mark.parametrize("T,k,E,N,kind,skip", CASES)
def test_permute_backward(T, k, E, N, kind, skip, dtype, out_dtype):
    rng, _, (off, srt, p2s, _) = tables(2, T, k, E, kind, skip)
    d = values(rng, (T * k, N), dtype)
    d[int(off[-1]):] = float("nan")            # rows of no pair are not read
    got = host(mq.moe_permute_backward(d, dev(p2s), k, out_dtype=out_dtype))
    dh = np.nan_to_num(host(d))
    ref = oracle.permute_backward(dh, p2s, k)
    mag = oracle.permute_backward(np.abs(dh), p2s, k)
    assert np.all(np.abs(got - ref) <= half_step(ref, out_dtype) + k * 2.0 ** -24 * mag)
    assert np.all(got[(p2s.reshape(T, k) < 0).all(1)] == 0)


@pytest.mark.parametrize("dout_dtype,y_dtype", [(F16, F16), (BF16, BF16), (F32, F32), (F32, BF16), (BF16, F16)])
@pytest.mark.parametrize("T,k,E,N,kind,skip", CASES)
def test_combine_backward(T, k, E, N, kind, skip, dout_dtype, y_dtype):
    rng, _, (off, srt, p2s, _) = tables(3, T, k, E, kind, skip)
    n = int(off[-1])
    dout, y = values(rng, (T, N), dout_dtype), values(rng, (T * k, N), y_dtype)
    y[n:] = float("nan")
    w = synth.softmax_weights(rng, T, k)
    dy = torch.full((T * k, N), 5, dtype=y_dtype, device="cuda")
    dw = torch.full((T, k), 5.0, device="cuda")
    got = mq.moe_scatter_combine_backward(dout, y, dev(p2s), dev(w), dy=dy, dw=dw)
    assert got[0] is dy and got[1] is dw
    dh, yh = host(dout), np.nan_to_num(host(y))
    rdy, rdw = oracle.scatter_combine_backward(dh, yh, p2s, w)
    _, mag = oracle.scatter_combine_backward(np.abs(dh), np.abs(yh), p2s, w)
    a = host(dy)
    assert np.all(a[n:] == 5)
    assert np.all(np.abs(a - rdy)[:n] <= (half_step(rdy, y_dtype) + 2.0 ** -24 * np.abs(rdy))[:n])
    b = host(dw)
    assert np.all(np.abs(b - rdw) <= half_step(rdw, F32) + (max(8, N / 256) + 16) * 2.0 ** -24 * mag)
    assert np.all(b.reshape(-1)[p2s < 0] == 0)


@pytest.mark.parametrize("T", [40, 1500])
def test_gradients_against_differences_of_the_forward_calls(T):
    """The combine is linear in y and in the weights, the permutation in x:
    <dout, f(v + d) - f(v - d)> / 2 = <gradient, d> with no truncation.  In
    fp32 both sides carry a few roundings (2^-24 each) of the sums of the
    magnitudes over T*k*N products; sums on the host in float64."""
    k, E, N = 3, 11, 136
    rng, _, (off, srt, p2s, _) = tables(4, T, k, E, "repeat", 0.2)
    n, P, p2 = int(off[-1]), T * k, dev(p2s)
    y, dout, w = values(rng, (P, N), F32), values(rng, (T, N), F32), dev(synth.softmax_weights(rng, T, k))
    diry, dirw, x, dirx = values(rng, (P, N), F32), values(rng, (T, k), F32), values(rng, (T, N), F32), values(rng, (T, N), F32)
    dy, dw = mq.moe_scatter_combine_backward(dout, y, p2, w)
    dot = lambda a, b: float((a.double() * b.double()).sum())
    mag = lambda a, b: float((a.double().abs() * b.double().abs()).sum())
    diff = lambda f, v, d: (f(v + d).double() - f(v - d).double()) / 2
    f = lambda v: mq.moe_scatter_combine(v, p2, w)
    lhs, rhs = dot(dout, diff(f, y, diry)), dot(dy[:n], diry[:n])
    assert abs(lhs - rhs) <= 64 * 2.0 ** -24 * (mag(dout, f(y.abs() + diry.abs())) + mag(dy[:n], diry[:n]))
    f = lambda v: mq.moe_scatter_combine(y, p2, v)
    lhs, rhs = dot(dout, diff(f, w, dirw)), dot(dw, dirw)
    m = mag(dout, mq.moe_scatter_combine(y.abs(), p2, w + dirw.abs()))
    assert abs(lhs - rhs) <= 64 * 2.0 ** -24 * (m + mag(dw, dirw))
    g = values(rng, (P, N), F32)
    lhs = dot(g[:n], diff(lambda v: mq.moe_permute(v, p2, k)[:n], x, dirx))
    rhs = dot(mq.moe_permute_backward(g, p2, k), dirx)
    m = mag(g[:n], mq.moe_permute(x.abs() + dirx.abs(), p2, k)[:n])
    assert abs(lhs - rhs) <= 64 * 2.0 ** -24 * (m + mag(mq.moe_permute_backward(g.abs(), p2, k), dirx))


def test_infinite_rows_stay_in_their_own_pairs():
    T, k, E, N = 20, 2, 4, 64
    rng, _, (off, srt, p2s, _) = tables(5, T, k, E)
    dout, y, w = values(rng, (T, N), F16), values(rng, (T * k, N), F16), synth.softmax_weights(rng, T, k)
    dy0, dw0 = mq.moe_scatter_combine_backward(dout, y, dev(p2s), dev(w))
    y[p2s[7]] = float("inf")                   # pair 7 = token 3, slot 1
    dy1, dw1 = mq.moe_scatter_combine_backward(dout, y, dev(p2s), dev(w))
    keep = torch.ones(T * k, dtype=torch.bool, device="cuda")
    keep[7] = False
    assert torch.equal(dw0.view(-1)[keep], dw1.view(-1)[keep]) and not torch.isfinite(dw1.view(-1)[7])
    assert torch.equal(dy0, dy1)


def test_offsets_past_32_bits():
    """More than 2^31 elements of sorted rows (4.5 GB of bf16)."""
    T, k, N = 17500, 4, 32768
    p2s = torch.from_numpy(np.random.default_rng(6).permutation(T * k).astype(np.int32)).cuda()
    x = torch.randn(T, N, device="cuda", dtype=BF16)
    xs = mq.moe_permute(x, p2s, k)
    assert xs.numel() > 2 ** 31
    for t in (0, 1, T // 2, T - 1):
        for j in range(k):
            assert torch.equal(xs[p2s[t * k + j].long()], x[t])
    dx = mq.moe_permute_backward(xs, p2s, k)
    assert torch.equal(dx, (x.float() * 4).to(BF16))   # four equal terms: exact
    w = torch.rand(T, k, device="cuda")
    dy, dw = mq.moe_scatter_combine_backward(x, xs, p2s, w)
    last = int(p2s.argmax())                            # the pair of the last sorted row
    t = last // k
    assert torch.equal(dy[-1], (x[t].float() * w.view(-1)[last]).to(BF16))
    ref = x[t].double().square().sum()
    assert abs(float(dw.view(-1)[last] - ref)) <= (N / 256 + 16) * 2.0 ** -24 * float(ref)


def test_more_tokens_than_one_grid_holds():
    """Past 2^23 workgroups every call goes out in runs of tokens; rows are
    powers of two, so every result is exact."""
    T, k, N = 2 ** 23 + 77, 2, 8
    P = T * k
    g = torch.Generator(device="cuda").manual_seed(55)
    p2s = torch.randperm(P, generator=g, device="cuda").int()
    p2s[torch.arange(0, P, 5, device="cuda")] = -1
    pairs = (p2s >= 0).nonzero().view(-1)
    s, t = p2s[pairs].long(), torch.div(pairs, k, rounding_mode="floor")
    two = lambda *shape: torch.randint(-3, 4, shape, generator=g, device="cuda").float().exp2()
    x, w, y = two(T, N).to(F16), two(T, k), two(P, N).to(F16)
    xs = torch.full((P, N), 7.0, dtype=F16, device="cuda")
    want = xs.clone()
    want[s] = x[t]
    assert torch.equal(mq.moe_permute(x, p2s, k, out=xs), want)
    both = torch.where((p2s >= 0)[:, None], y[p2s.clamp(min=0).long()], 0).view(T, k, N)
    assert torch.equal(mq.moe_permute_backward(y, p2s, k), both[:, 0] + both[:, 1])
    wide = both.float() * w[:, :, None]
    assert torch.equal(mq.moe_scatter_combine(y, p2s, w, out_dtype=F32),
                       wide[:, 0] + wide[:, 1])
    dy, dw = mq.moe_scatter_combine_backward(x, y, p2s, w, dy=torch.full_like(y, 7.0))
    want.fill_(7.0)
    want[s] = (x[t].float() * w.view(-1)[pairs, None]).to(F16)
    assert torch.equal(dy, want)
    assert torch.equal(dw, (both.float() * x[:, None].float()).sum(2))
