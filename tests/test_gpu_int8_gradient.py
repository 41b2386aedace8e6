"""The INT8 product's gradient keeps the bits of its fp32 formula, and takes its
rows in parts where the workspace is small.

Tolerance per element, u = 2^-24: d = dy * w_scale is one fp32 rounding, its
code two more (the factor 8355711 / max and the product), the step one: 4 u |d|
and half a step, step = max|d| / 8355711.  The three sums are exact; a digit's
sum, brought to its place, is at most mag + 0x8080 step sum|w| (a digit rounds
what is below it to the nearest), so that their conversions and the two joins, 5
u of it, add 5 u mag and 0.01 step sum|w|; the last join is one rounding more:
(0.51 step) sum|w| + 10 u mag + u |base|, and half a step of the output."""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import dev, host
from tests.test_gpu_int8 import GRADS, U, Experts, grad_case, within
from tests.test_gpu_permute import BF16, F16, half_step

pytestmark = pytest.mark.gpu

mq = pytest.importorskip("quantized_moe_grouped_route_amd")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mq.lib()


def tolerance(r, dtype, base=0.0):
    return (half_step(r["dx"], dtype) + 0.51 / 8355711 * r["top"][:, None] * r["wsum"] + 10 * U * r["mag"] +
            U * np.abs(base))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("N,K,rows", [(96, 128, 5), (288, 384, 130), (7168, 256, 40), (33024, 128, 9)])
@pytest.mark.parametrize("large", [1.0, 100.0, 3000.0])
def test_columns_beside_a_large_one_keep_their_bits(large, N, K, rows, dtype):
    # one column of d far above the others, with weights of zero in half of the outputs: these
    # hold what the other columns leave
    rng = np.random.default_rng(N + rows)
    w = rng.integers(-128, 128, (2, N, K)).astype(np.int8)
    col = N // 3
    w[:, col, ::2] = 0
    sw = ((rng.random((2, N)) + 0.5) / 64).astype(np.float32)
    sw[:, col] *= large
    dy = torch.from_numpy(rng.standard_normal((rows, N)).astype(np.float32)).to(dtype).cuda()
    off = np.array([0, rows // 3, rows])
    r = oracle.grouped_gemm_qint8_backward(host(dy), w, sw, off)
    dx = mq.grouped_gemm_qint8_backward(dy, dev(w), dev(sw), dev(off.astype(np.int32)))
    within(host(dx), r["dx"], tolerance(r, dtype))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("case", GRADS, ids=[f"T{c[0]}k{c[1]}E{c[2]}N{c[3]}K{c[4]}-{c[5]}" for c in GRADS])
def test_every_workspace_gives_the_same_bits(case, dtype):
    T, k, E, N, K, kind, skip = case
    p = Experts(31, T, k, E, N, K, "sorted", kind, skip)
    dy, b = grad_case(p, dtype, True)
    r = oracle.grouped_gemm_qint8_backward(np.nan_to_num(host(dy)), p.w, p.sw, p.off, host(b))
    least = mq.qint8_backward_workspace_bytes(p.P, E, N, K)
    most = mq.qint8_backward_workspace_bytes(p.P, E, N, K, at_once=True)
    assert least <= most
    first = None
    for size in sorted({least, (least + most) // 2, most}):
        ws = torch.full((size + 512,), 173, dtype=torch.uint8, device="cuda")
        dx = torch.full((p.P + 3, K), 7.0, dtype=dtype, device="cuda")
        mq.grouped_gemm_qint8_backward(dy, p.d["w"], p.d["sw"], p.d["off"], base=b, dx=dx[:p.P], workspace=ws[:size])
        first = dx if first is None else first
        assert torch.equal(dx, first)                             # rows of no expert and past P among them
        assert bool((dx[p.n:] == 7).all()) and bool((ws[size:] == 173).all())
    within(host(first)[:p.n], r["dx"][:p.n], tolerance(r, dtype, host(b))[:p.n])
    # a larger workspace than the largest that helps stays as it was behind that
    ws = torch.full((most + 4096,), 173, dtype=torch.uint8, device="cuda")
    dx = mq.grouped_gemm_qint8_backward(dy, p.d["w"], p.d["sw"], p.d["off"], base=b, workspace=ws)
    assert torch.equal(dx[:p.n], first[:p.n]) and bool((ws[most:] == 173).all())


@pytest.mark.parametrize("rows", [1, 2, 3, 64, 97])
def test_few_rows_in_the_least_workspace(rows):
    rng = np.random.default_rng(rows)
    E, N, K = 3, 160, 256
    w, sw = rng.integers(-128, 128, (E, N, K)).astype(np.int8), (rng.random((E, N)) + 0.5).astype(np.float32)
    off = np.array([0, rows // 2, rows // 2, rows])
    dy = torch.from_numpy(rng.standard_normal((rows, N)).astype(np.float32)).to(BF16).cuda()
    ws = torch.full((mq.qint8_backward_workspace_bytes(rows, E, N, K),), 255, dtype=torch.uint8, device="cuda")
    dx = mq.grouped_gemm_qint8_backward(dy, dev(w), dev(sw), dev(off.astype(np.int32)), workspace=ws)
    r = oracle.grouped_gemm_qint8_backward(host(dy), w, sw, off)
    within(host(dx), r["dx"], tolerance(r, BF16))
    for i in range(rows):                                         # each row alone: the same bits
        e = int(np.searchsorted(off, i, side="right")) - 1
        one = np.zeros(E + 1, np.int32)
        one[e + 1:] = 1
        assert torch.equal(mq.grouped_gemm_qint8_backward(dy[i:i + 1].clone(), dev(w), dev(sw), dev(one)), dx[i:i + 1])


def test_two_parts_captured_and_replayed():
    from tests.test_gpu_graphs import _capture_and_replay
    p = Experts(32, 700, 2, 7, 544, 384, "sorted", "repeat", 0.1)
    dy, b = grad_case(p, F16, True)
    ws = torch.zeros(mq.qint8_backward_workspace_bytes(p.P, 7, 544, 384), dtype=torch.uint8, device="cuda")
    dx = torch.zeros(p.P, 384, dtype=F16, device="cuda")

    def step():
        mq.grouped_gemm_qint8_backward(dy, p.d["w"], p.d["sw"], p.d["off"], base=b, dx=dx, workspace=ws)
    _capture_and_replay(step, [dx[:p.n]])
