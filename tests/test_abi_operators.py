"""What the permutation, combine-gradient and adapter calls take and refuse at
their limits (no GPU needed; the C calls see addresses only)."""
import pytest

import quantized_moe_grouped_route_amd as mq
from tests.test_abi_lora import L, _lora, _lora_bwd  # noqa: F401  (L: the library, a fixture)


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
