"""The permutation, gradient and adapter calls at the limits that they take."""
import numpy as np
import pytest
import torch

from tests.gpu_util import dev, host
from tests.test_gpu_lora import close, values
from tests.test_gpu_permute import BF16, F16, tables

pytestmark = pytest.mark.gpu

mq = pytest.importorskip("quantized_moe_grouped_route_amd")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mq.lib()


def test_forward_of_many_wide_groups_of_a_high_rank():
    """1024 groups, 16384 -> 16384 at rank 256: sizes whose gradients are refused.
    9 GB of each weight; the groups without rows are not read."""
    E, N, K, R, P = 1024, 16384, 16384, 256, 5
    rng = np.random.default_rng(71)
    off = np.zeros(E + 1, np.int32)
    off[1:] = 2
    off[E] = P
    used = [0, 0, E - 1, E - 1, E - 1]
    a = torch.full((E, R, K), float("nan"), dtype=BF16, device="cuda")
    b = torch.full((E, N, R), float("nan"), dtype=BF16, device="cuda")
    for e in (0, E - 1):
        a[e], b[e] = values(rng, (R, K), BF16, K ** -0.5), values(rng, (N, R), BF16, R ** -0.5)
    x, base = values(rng, (P, K), BF16), values(rng, (P, N), BF16)
    out = host(mq.grouped_lora(x, a, b, dev(off), None, 1, a_row="sorted", base=base))
    for s, e in enumerate(used):
        ah, bh, xh, bs = host(a[e]), host(b[e]), host(x[s]), host(base[s])
        close(out[s], bs + bh @ (ah @ xh), np.abs(bs) + np.abs(bh) @ (np.abs(ah) @ np.abs(xh)), BF16, (K, N, R, P), s)


def test_forward_of_more_rows_than_the_gradients_take():
    """2^26 + 5 rows of 8: one row in every 4099, and the last ones."""
    P, N, K, R = 2 ** 26 + 5, 8, 8, 8
    rng = np.random.default_rng(72)
    off = np.array([0, P // 3, P - 2], np.int32)
    g = torch.Generator(device="cuda").manual_seed(72)
    x = torch.randn(P, K, generator=g, device="cuda").to(F16)
    a, b = values(rng, (2, R, K), F16, 0.3), values(rng, (2, N, R), F16, 0.3)
    out = torch.full((P, N), 7.0, dtype=F16, device="cuda")
    mq.grouped_lora(x, a, b, dev(off), None, 1, a_row="sorted", out=out)
    s = np.unique(np.concatenate([np.arange(0, P, 4099), np.arange(P - 40, P)]))
    pick = torch.from_numpy(s).cuda()
    xh, got = host(x[pick]), host(out[pick])
    for e in (0, 1):
        i = (s >= off[e]) & (s < off[e + 1])
        h, m = xh[i] @ host(a[e]).T, np.abs(xh[i]) @ np.abs(host(a[e])).T
        close(got[i], h @ host(b[e]).T, m @ np.abs(host(b[e])).T, F16, (K, N, R), e)
    assert np.all(got[s >= off[2]] == 7)


def test_combine_gradient_of_y_with_spare_rows():
    """Buffers of a larger batch: the rows past T*topk are neither read nor
    written, and the results are those of the exact sizes."""
    T, k, E, N = 37, 3, 5, 264
    rng, _, (off, _, p2s, _) = tables(73, T, k, E, "repeat", 0.2)
    dout, y, w = values(rng, (T, N), BF16), values(rng, (T * k + 9, N), BF16), dev(rng.random((T, k)).astype(np.float32))
    y[int(off[-1]):] = float("nan")
    dy0, dw0 = mq.moe_scatter_combine_backward(dout, y[:T * k], dev(p2s), w)
    n = int(off[-1])
    for rows in (T * k + 9, T * k):
        dy = torch.full((rows, N), 7.0, dtype=BF16, device="cuda")
        got, dw = mq.moe_scatter_combine_backward(dout, y, dev(p2s), w, dy=dy)
        assert got is dy and torch.equal(dw, dw0)
        assert torch.equal(dy[:n], dy0[:n]) and torch.all(dy[n:] == 7)
