"""The INT8 product at the most rows that a call can name."""
import pytest
import torch

pytestmark = pytest.mark.gpu

mq = pytest.importorskip("quantized_moe_grouped_route_amd")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mq.lib()


@pytest.mark.parametrize("sched", ["prefill", "decode"])
def test_one_expert_of_the_most_rows(sched):
    """2^31 - 1 pairs of 2^25 tokens, all of one expert: the rows round up to whole
    tiles past 2^31.  82 GB: 69 of outputs, 9 of pair ids, 4 of activations."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free device memory")
    P, T, k, N, K = 2 ** 31 - 1, 2 ** 25, 64, 32, 128
    g = torch.Generator(device="cuda").manual_seed(61)
    w = torch.randint(-128, 128, (1, N, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.full((1, N), 2.0 ** -14, device="cuda")
    a = torch.randint(-128, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    sa = torch.full((T,), 2.0 ** -4, device="cuda")
    srt = torch.arange(P, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    out = torch.full((P, N // 2), float("nan"), dtype=torch.float16, device="cuda")
    mq.grouped_gemm_qint8(a, sa, w, sw, off, srt, k, act="silu_mul", out=out, sched=sched)
    # a token's slots hold the same row
    some = torch.tensor([0, 1, 77, T // 2, T - 2, T - 1], device="cuda")
    few = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    ref = mq.grouped_gemm_qint8(a[some].contiguous(), sa[:6].clone(), w, sw, few, None, 1, act="silu_mul")
    for i, t in enumerate(some.tolist()):
        rows = out[k * t:min(P, k * t + k)]
        assert torch.equal(rows, ref[i].expand_as(rows)), t
    for lo in range(0, P, 2 ** 27):                               # every row is written
        assert not bool(torch.isnan(out[lo:lo + 2 ** 27, 0]).any())
    del a, srt, out
    torch.cuda.empty_cache()
