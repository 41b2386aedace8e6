"""What the permutation, combine-gradient and adapter calls take and refuse at
their limits (no GPU needed; the C calls see addresses only)."""
import pytest
import torch

import quantized_moe_grouped_route_amd as mq
from tests.test_abi_lora import L, _combine_bwd, _lora, _lora_bwd, _permute, _permute_bwd, at  # noqa: F401  (L: the library, a fixture)


# Many wide groups of a high rank: the gradients' weight sums need more
# workgroups than one launch holds, the forward call's two products do not.
@pytest.mark.parametrize("P", [1, 4096])
def test_the_forward_call_has_its_own_size_limit(L, P):
    kw = dict(P=P, E=1024, N=16384, K=16384, R=256, rows=P, arow=1, topk=1, wsb=1 << 40)
    assert L.grouped_lora_workspace_bytes(P, 1024, 16384, 16384, 256) >= P * 256 * 4
    assert _lora(L, **kw, out=None) == mq.EINVAL        # refused for out, not for the sizes
    assert b"null pointer" in L.moeq_last_error()
    assert L.grouped_lora_backward_workspace_bytes(P, 1024, 16384, 16384, 256) == 0
    assert _lora_bwd(L, **kw) == mq.EINVAL
    assert b"too large for one launch" in L.moeq_last_error()


def test_the_forward_call_takes_more_rows_than_its_gradients(L):
    P = 2 ** 26
    assert L.grouped_lora_workspace_bytes(P, 1, 8, 8, 8) == P * 8 * 4
    assert L.grouped_lora_backward_workspace_bytes(P, 1, 8, 8, 8) == 0
    assert L.grouped_lora_workspace_bytes(2 * P, 1, 8, 8, 8) == 0


# The tables and the scales are inputs too: an output over one of them would
# change them while the call reads them.
@pytest.mark.parametrize("out", ["out", "h", "ws"])
@pytest.mark.parametrize("table,nbytes", [("sc", 4 * 4), ("off", 5 * 4), ("srt", 16 * 4), ("p2s", 16 * 4)])
def test_lora_refuses_outputs_over_the_tables(L, out, table, nbytes):
    kw = dict(p2s=at(12), orow=1, h=at(9))
    where = dict(sc=at(3), off=at(4), srt=at(5), p2s=at(12))[table]
    need = L.grouped_lora_workspace_bytes(16, 4, 64, 8192, 16)
    size = dict(out=16 * 64 * 2, h=16 * 16 * 4, ws=need)[out]
    for p in (where, where + (nbytes - 1) // 16 * 16, where - (size - 1) // 16 * 16):
        assert _lora(L, **{**kw, out: p}) == mq.EINVAL
        assert b"overlaps" in L.moeq_last_error()


@pytest.mark.parametrize("out", ["dx", "da", "db", "ws"])
@pytest.mark.parametrize("table,nbytes", [("sc", 4 * 4), ("off", 5 * 4), ("srt", 16 * 4)])
def test_lora_backward_refuses_outputs_over_the_tables(L, out, table, nbytes):
    where = dict(sc=at(4), off=at(6), srt=at(7))[table]
    size = dict(dx=16 * 128 * 2, da=4 * 16 * 128 * 2, db=4 * 64 * 16 * 2,
                ws=L.grouped_lora_backward_workspace_bytes(16, 4, 64, 128, 16))[out]
    for p in (where, where + (nbytes - 1) // 16 * 16, where - (size - 1) // 16 * 16):
        assert _lora_bwd(L, **{out: p}) == mq.EINVAL
        assert b"overlaps" in L.moeq_last_error()


@pytest.mark.parametrize("call,out,size,table", [
    (_permute, "xs", 8 * 64 * 2, at(1)), (_permute_bwd, "dx", 4 * 64 * 4, at(1)),
    (_combine_bwd, "dy", 8 * 64 * 2, at(2)), (_combine_bwd, "dw", 8 * 4, at(2)),
])
def test_permutation_and_gradients_refuse_outputs_over_the_pair_table(L, call, out, size, table):
    for p in (table, table + 8 * 4 - 16, table - size + 16):
        assert call(L, **{out: p}) == mq.EINVAL
        assert b"overlaps" in L.moeq_last_error()


def test_combine_gradient_takes_y_with_spare_rows_where_dy_is_given():
    # (a workspace of a larger batch, as the forward call takes; refused here
    # for being on the CPU, not for its shape)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    p2s, w = torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2)
    for rows in (9, 8):
        with pytest.raises(ValueError, match="GPU"):
            mq.moe_scatter_combine_backward(bf(4, 64), bf(9, 64), p2s, w, dy=bf(rows, 64))
    with pytest.raises(ValueError, match="give dy"):
        mq.moe_scatter_combine_backward(bf(4, 64), bf(9, 64), p2s, w)
    with pytest.raises(ValueError, match="dy must be"):
        mq.moe_scatter_combine_backward(bf(4, 64), bf(9, 64), p2s, w, dy=bf(10, 64))
    with pytest.raises(ValueError, match="dy must be"):
        mq.moe_scatter_combine_backward(bf(4, 64), bf(8, 64), p2s, w, dy=bf(9, 64))
    with pytest.raises(ValueError, match="at least"):
        mq.moe_scatter_combine_backward(bf(4, 64), bf(7, 64), p2s, w, dy=bf(7, 64))
