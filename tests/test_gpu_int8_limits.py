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


def behind(rows, cols, dtype, fill):
    """A tensor of `rows` rows and the larger one that it leads, full of `fill`."""
    whole = torch.full((rows + 64, cols), fill, dtype=dtype, device="cuda")
    return whole[:rows], whole[rows:]


@pytest.mark.parametrize("off", [[0, 70, 20, 1000, 5000], [-5, 10, 9, 40, 2000000000], [0, 0, 0, 0, -7],
                                 [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1]])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_malformed_tables_write_nothing_behind_the_outputs(off, dtype):
    P, E, N, K, B = 80, 4, 96, 256, 1
    g = torch.Generator(device="cuda").manual_seed(62)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)
    w = torch.randint(-128, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand(E, N, generator=g, device="cuda")
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    dy, base, gu, dh = rnd(P, N), rnd(P, K), rnd(P, N), rnd(P, N // 2)
    for at_once in (False, True):
        ws, ws_tail = behind(mq.qint8_backward_workspace_bytes(P, E, N, K, at_once=at_once), 1, torch.uint8, 77)
        dx, dx_tail = behind(P, K, dtype, 7.0)
        mq.grouped_gemm_qint8_backward(dy, w, sw, o, base=base, dx=dx, workspace=ws.view(-1))
        assert bool((dx_tail == 7).all()) and bool((ws_tail == 77).all())
    (h, h_tail), (ck, ck_tail), (cs, cs_tail) = (behind(P, N // 2, dtype, 7.0), behind(P, N, torch.int8, 77),
                                                 behind(P, 2 * B, torch.float32, 7.0))
    mq.moe_silu_mul(gu, o, checkpoint=True, h=h, ck=ck, cs=cs)
    assert bool((h_tail == 7).all()) and bool((ck_tail == 77).all()) and bool((cs_tail == 7).all())
    for kw in (dict(gu=gu), dict(ck=ck, cs=cs)):
        (d, d_tail), (h, h_tail) = behind(P, N, dtype, 7.0), behind(P, N // 2, dtype, 7.0)
        mq.moe_silu_mul_backward(dh, o, need_h=True, dgu=d, h=h, **kw)
        assert bool((d_tail == 7).all()) and bool((h_tail == 7).all())
    h, h_tail = behind(P, N // 2, dtype, 7.0)
    mq.moe_silu_mul_again(ck, cs, o, dtype=dtype, h=h)
    assert bool((h_tail == 7).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_h_alone_from_the_columns(dtype):
    # the C entry takes gu, without dh and dgu: the bits of the forward call
    P, I, E = 70, 200, 3
    g = torch.Generator(device="cuda").manual_seed(63)
    gu = (3 * torch.randn(P, 2 * I, generator=g, device="cuda")).to(dtype)
    off = torch.tensor([0, 10, 10, 61], dtype=torch.int32, device="cuda")
    h = torch.full((P, I), 7.0, dtype=dtype, device="cuda")
    st = mq.lib().moe_silu_mul_backward(None, mq._DTYPE_CODE[dtype], gu.data_ptr(), None, None, off.data_ptr(), E, P, I,
                                        None, h.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == mq.OK, mq.lib().moeq_last_error()
    ref = mq.moe_silu_mul(gu, off)[0]
    assert torch.equal(h[:61], ref[:61]) and bool((h[61:] == 7).all())
