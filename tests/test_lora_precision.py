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
