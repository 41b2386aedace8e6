"""Workspace sizes of the INT8 product's gradient (no GPU needed)."""
import pytest

import quantized_moe_grouped_route_amd as mq
from tests.test_abi_int8 import _grad
from tests.test_abi_lora import L, at  # noqa: F401  (L: the library, a fixture)


@pytest.mark.parametrize("P,N,least,most", [
    (0, 64, 0, 0), (1, 32, 3 * 128 + 4, 3 * 128 + 4), (2, 32, 2 * 260, 2 * 388), (1, 160, 3 * 256 + 4, 3 * 256 + 4),
    (1000, 128, 260000, 388000), (16, 160, 16 * 516, 16 * 772),
])
def test_workspace_of_one_row_and_of_all(L, P, N, least, most):  # noqa: F811
    assert L.grouped_gemm_qint8_backward_workspace_bytes(P, 4, N, 128) == least
    assert mq.qint8_backward_workspace_bytes(P, 4, N, 128) == least
    assert mq.qint8_backward_workspace_bytes(P, 4, N, 128, at_once=True) == most
    assert mq.qint8_backward_workspace_bytes(P, 4, 48, 128, at_once=True) == 0      # N no multiple of 32


def test_workspace_that_is_used_may_not_overlap(L):  # noqa: F811
    # 16 rows of 64: at most 16 * 388 bytes are used, whatever is given
    at_dx = at(5)
    assert _grad(L, ws=at_dx - 16 * 388 + 16) == mq.EINVAL
    assert _grad(L, ws=at_dx - 16 * 260 - 16, wsb=16 * 388) == mq.EINVAL
    assert _grad(L, P=1, wsb=387) == mq.EINVAL and b"388 bytes needed" in L.moeq_last_error()
