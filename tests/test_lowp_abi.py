"""Refusals of the low-precision entry points, all before anything is
launched (no GPU here), and the size of the scales."""
import math

import pytest

from fp64_gemm_emulation_exponent_gb300 import build as ozk_build
from fp64_gemm_emulation_exponent_gb300 import ozk

BIG = 1 << 44  # addresses that nothing dereferences, far apart
A, B, C, D, E, OFF = (BIG * i for i in range(1, 7))


@pytest.fixture(scope="module", autouse=True)
def built_library():
    ozk_build.build()
    yield


def quantize(rows=4, K=64, X=A, ldx=None, dtype=0, fmt=0, prescale=1.0, offsets=None, groups=1, codes=B, scales=C):
    return ozk.lib().ozk_mx4_quantize(rows, K, X, K if ldx is None else ldx, dtype, fmt, prescale, offsets, groups, codes,
                                      scales, None)


def dequantize(rows=4, K=64, codes=B, scales=C, fmt=0, offsets=None, groups=1, X=A, ldx=None, dtype=0):
    return ozk.lib().ozk_mx4_dequantize(rows, K, codes, scales, fmt, offsets, groups, X, K if ldx is None else ldx, dtype,
                                        None)


def product(T=4, N=8, K=64, groups=1, offsets=None, xc=A, xs=B, wc=C, ws=D, fmt=0, Y=E, ldy=None, out=0):
    return ozk.lib().ozk_mx4_grouped_gemm(T, N, K, groups, offsets, xc, xs, wc, ws, fmt, 1.0, Y, N if ldy is None else ldy,
                                          out, None)


def forward(T=4, N=8, K=64, groups=2, offsets=OFF, X=A, ldx=None, W=B, ldw=None, stride=None, dtype=0, Y=C, ldy=None, out=0,
            name="ozk_grouped_gemm"):
    rows, cols = (K, N) if name == "ozk_grouped_gemm" else (N, K)
    ldw = K if ldw is None else ldw
    return getattr(ozk.lib(), name)(T, N, K, groups, offsets, X, rows if ldx is None else ldx, W, ldw,
                                    N * ldw if stride is None else stride, dtype, Y, cols if ldy is None else ldy, out, None)


def grad_w(T=4, N=8, K=64, groups=2, offsets=OFF, dY=A, lddy=None, X=B, ldx=None, dtype=0, W=C, ldw=None, stride=None, out=0):
    ldw = K if ldw is None else ldw
    return ozk.lib().ozk_grouped_gemm_dw(T, N, K, groups, offsets, dY, N if lddy is None else lddy, X,
                                         K if ldx is None else ldx, dtype, W, ldw, N * ldw if stride is None else stride, out,
                                         None)


INVALID, UNSUPPORTED = ozk.OZK_ERR_INVALID_ARG, ozk.OZK_ERR_UNSUPPORTED


def test_scale_bytes():
    for fmt, span in (("nvfp4", 64), ("mxfp4", 128)):
        f = {"nvfp4": ozk.OZK_NVFP4, "mxfp4": ozk.OZK_MXFP4}[fmt]
        for rows, K, groups in ((1, 1, 1), (127, 64, 1), (128, 65, 1), (129, 1000, 1), (5000, 4096, 7), (0, 64, 3)):
            want = (rows // 128 + groups) * math.ceil(math.ceil(K / 64) * 64 / span) * 512
            assert ozk.lib().ozk_mx4_scale_bytes(rows, K, f, groups) == want
            assert ozk.mx4_scale_bytes(rows, K, fmt, groups) == want
    for bad in ((-1, 64, 0, 1), (1, -1, 0, 1), (1, 64, 2, 1), (1, 64, 0, 0), (1, 64, 0, 1025), (1 << 40, 64, 0, 1)):
        assert ozk.lib().ozk_mx4_scale_bytes(*bad) == 0


def test_every_group_has_room_for_its_scales():
    """Row block o / 128 + g of a group never lies below the end of the group before it."""
    for counts in ([0, 0, 1], [127, 1, 128, 129], [1] * 300, [128] * 5, [255, 1, 1, 0, 640]):
        o, end = 0, 0
        for g, c in enumerate(counts):
            assert o // 128 + g >= end
            end = o // 128 + g + -(-c // 128)
            o += c
        assert end <= o // 128 + len(counts)


@pytest.mark.parametrize("call", [quantize, dequantize])
def test_matrix_refusals(call):
    for bad in (dict(rows=-1), dict(K=-1), dict(fmt=2), dict(groups=0), dict(rows=5, groups=2), dict(dtype=4), dict(dtype=-1),
                dict(X=None), dict(codes=None), dict(scales=None), dict(ldx=63), dict(codes=B + 8), dict(scales=C + 4),
                dict(X=A + 1), dict(codes=A), dict(scales=A)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(rows=1 << 31), dict(K=(1 << 22) + 1), dict(groups=1025, offsets=OFF)):
        assert call(**bad) == UNSUPPORTED, bad
    for empty in (dict(rows=0), dict(K=0), dict(rows=0, X=None, codes=None, scales=None)):
        assert call(**empty) == ozk.OZK_OK


def test_quantize_prescale_refusals():
    for p in (0.0, -1.0, math.inf, math.nan):
        assert quantize(prescale=p) == INVALID


def test_product_refusals():
    for bad in (dict(T=-1), dict(N=-1), dict(K=-1), dict(fmt=3), dict(groups=0), dict(groups=2), dict(Y=None), dict(ldy=7),
                dict(Y=E + 1), dict(Y=E + 2, out=2), dict(xc=None), dict(xs=None), dict(wc=None), dict(ws=None), dict(xc=A + 8),
                dict(ws=D + 2), dict(Y=A), dict(Y=D)):
        assert product(**bad) == INVALID, bad
    for bad in (dict(out=3), dict(out=7), dict(T=1 << 31), dict(N=1 << 23), dict(K=1 << 23), dict(groups=1025, offsets=OFF),
                dict(N=1 << 22, groups=1000, offsets=OFF)):
        assert product(**bad) == UNSUPPORTED, bad
    for empty in (dict(T=0), dict(N=0)):
        assert product(**empty) == ozk.OZK_OK
    assert ozk.lib().ozk_mx4_gemm(-1, 8, 64, A, B, C, D, 0, 1.0, E, 8, 0, None) == INVALID


@pytest.mark.parametrize("name", ["ozk_grouped_gemm", "ozk_grouped_gemm_dx"])
def test_grouped_refusals(name):
    call = lambda **k: forward(name=name, **k)  # noqa: E731
    for bad in (dict(T=-1), dict(N=-1), dict(K=-1), dict(groups=0), dict(offsets=None), dict(X=None), dict(W=None),
                dict(Y=None), dict(ldx=0), dict(ldw=56), dict(ldy=7), dict(stride=8 * 64 - 8), dict(Y=C + 1),
                dict(Y=C + 2, out=2), dict(Y=A), dict(Y=B)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dtype=2), dict(dtype=3), dict(out=1), dict(out=3), dict(X=A + 8), dict(W=B + 2), dict(ldx=68), dict(ldw=68),
                dict(stride=8 * 64 + 4), dict(T=1 << 31), dict(N=1 << 23), dict(K=1 << 23), dict(groups=1025)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(T=0) == ozk.OZK_OK


def test_grad_w_refusals():
    for bad in (dict(T=-1), dict(offsets=None), dict(dY=None), dict(X=None), dict(W=None), dict(lddy=0), dict(ldx=56),
                dict(ldw=56), dict(stride=504), dict(W=A), dict(W=B), dict(W=C + 1)):
        assert grad_w(**bad) == INVALID, bad
    for bad in (dict(dtype=2), dict(out=1), dict(dY=A + 2), dict(X=B + 8), dict(lddy=12), dict(ldx=68), dict(groups=2000)):
        assert grad_w(**bad) == UNSUPPORTED, bad
    assert grad_w(N=0) == ozk.OZK_OK
