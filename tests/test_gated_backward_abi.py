"""The whole backward pass of the gated product refuses a call before it
launches anything (no GPU here: a call that is not refused ends at the device)."""
import pytest

from fp64_gemm_emulation_exponent_gb300 import build as ozk_build
from fp64_gemm_emulation_exponent_gb300 import ozk

BIG = 1 << 50  # addresses that nothing dereferences, far apart
X, W, S, P, DH, DX, DW, OFF = (BIG * i for i in range(1, 9))
INVALID, UNSUPPORTED = ozk.OZK_ERR_INVALID_ARG, ozk.OZK_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built_library():
    ozk_build.build()
    yield


def backward(T=4, N=8, K=64, groups=2, x=X, w=W, p=P, dx=DX, dw=DW):
    return ozk.lib().ozk_grouped_gated_gemm_grad(T, N, K, groups, OFF, DH, N, S, N, T * N, x, K, w, K, 2 * N * K, 0, p, 2 * N,
                                                 dx, K, dw, K, 2 * N * K, None)


def test_a_result_on_an_odd_address():
    assert backward(dx=DX + 1) == INVALID
    assert backward(dw=DW + 1) == INVALID


def test_more_tiles_than_the_products_count():
    many = dict(T=1 << 30, K=1 << 16, groups=1)  # dX: 2^23 by 2^9 tiles
    assert backward(**many) == UNSUPPORTED
    assert backward(**many, dw=None) == UNSUPPORTED
    assert backward(T=4, N=1 << 18, K=1 << 16, groups=1024) == UNSUPPORTED  # dW: 2^12 by 2^10 by 2^9
    assert backward(T=4, N=1 << 18, K=1 << 16, groups=1024, dx=None) == UNSUPPORTED


def test_results_over_operands_of_empty_products():
    """Without columns dX is cleared all the same, and without rows dW: neither may lie on what is read elsewhere."""
    for bad in (dict(N=0, dx=X), dict(N=0, dx=X + 64), dict(T=0, dw=W), dict(T=0, dw=W + 2)):
        assert backward(**bad) == INVALID, bad


def test_empty_operands_lie_over_nothing():
    """Memory of no bytes may have any address, one inside a result too: no refusal (the call ends at the device)."""
    for fine in (dict(T=0, x=DW + 64, dx=DW + 64), dict(N=0, dw=DX + 64, w=DX + 64, p=DX + 64), dict(K=0, x=P + 2, w=P + 4)):
        assert backward(**fine) not in (INVALID, UNSUPPORTED), fine
