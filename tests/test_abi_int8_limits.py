"""The sizes that the INT8 calls take end where their headers say (no GPU needed):
nothing is launched, a call inside the limits is refused for another argument."""
import pytest

import quantized_moe_grouped_route_amd as mq
from tests.test_abi_int8 import _gemm, _grad
from tests.test_abi_lora import L, at  # noqa: F401  (L: the library, a fixture)

MANY = 1 << 20     # (P/16 + E) * 1024 = 2^30 with N = 16384, (P/32 + E) * 1024 with K = 131072


@pytest.mark.parametrize("K", [128, 4096, 65536, 131072 - 128])
@pytest.mark.parametrize("rows,E,inside", [((MANY - 8) * 16, 8, False), ((MANY - 8) * 16 - 1, 8, True),
                                           ((MANY - 1024) * 16, 1024, False), ((MANY - 1024) * 16 - 1, 1024, True),
                                           (1 << 21, 8, True)])
def test_items_of_the_product(L, rows, E, inside, K):  # noqa: F811
    assert _gemm(L, P=rows, rows=rows, E=E, N=16384, K=K, out=at(0)) == mq.EINVAL
    text = L.moeq_last_error()
    assert (b"overlaps" in text) == inside and (b"too large" in text) != inside


@pytest.mark.parametrize("N", [32, 4096, 131072 - 32])
@pytest.mark.parametrize("rows,E,inside", [((MANY - 8) * 32, 8, False), ((MANY - 8) * 32 - 1, 8, True),
                                           ((MANY - 1024) * 32, 1024, False), ((MANY - 1024) * 32 - 1, 1024, True)])
def test_items_of_the_gradient(L, rows, E, inside, N):  # noqa: F811
    K = 131072
    assert (L.grouped_gemm_qint8_backward_workspace_bytes(rows, E, N, K) > 0) == inside
    assert _grad(L, P=rows, E=E, N=N, K=K, dx=at(0), wsb=1 << 60) == mq.EINVAL
    text = L.moeq_last_error()
    assert (b"overlaps" in text) == inside and (b"too large" in text) != inside
