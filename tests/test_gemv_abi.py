"""Refusals of the products of a few rows with 4-bit weights, all before
anything is launched (no GPU here), and the rule on their source."""
import os
import re

import pytest

from fp64_gemm_emulation_exponent_gb300 import build as ozk_build
from fp64_gemm_emulation_exponent_gb300 import ozk

BIG = 1 << 44  # addresses that nothing dereferences, far apart
A, B, C, D, OFF = (BIG * i for i in range(1, 6))
INVALID, UNSUPPORTED = ozk.OZK_ERR_INVALID_ARG, ozk.OZK_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built_library():
    ozk_build.build()
    yield


def plain(T=4, N=8, K=64, groups=1, offsets=None, X=A, ldx=None, dtype=0, wc=B, ws=C, fmt=0, alpha=1.0, Y=D, ldy=None, out=0):
    return ozk.lib().ozk_mx4_gemv(T, N, K, groups, offsets, X, K if ldx is None else ldx, dtype, wc, ws, fmt, alpha, Y,
                                  N if ldy is None else ldy, out, None)


def gated(T=4, N=8, K=64, groups=1, offsets=None, X=A, ldx=None, dtype=0, wc=B, ws=C, fmt=0, alpha=1.0, act=0, Y=D, ldy=None,
          out=0):
    return ozk.lib().ozk_mx4_gated_gemv(T, N, K, groups, offsets, X, K if ldx is None else ldx, dtype, wc, ws, fmt, alpha,
                                        act, Y, N if ldy is None else ldy, out, None)


@pytest.mark.parametrize("call", [plain, gated])
def test_refusals(call):
    for bad in (dict(T=-1), dict(N=-1), dict(K=-1), dict(fmt=2), dict(fmt=-1), dict(groups=0), dict(groups=2), dict(X=None),
                dict(wc=None), dict(ws=None), dict(Y=None), dict(ldx=63), dict(ldy=7), dict(X=A + 1), dict(wc=B + 8),
                dict(ws=C + 4), dict(Y=D + 1), dict(Y=D + 2, out=2), dict(Y=A), dict(Y=B), dict(Y=C)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dtype=2), dict(dtype=3), dict(out=3), dict(T=1 << 31), dict(K=(1 << 22) + 1), dict(N=(1 << 22) + 1),
                dict(groups=1025, offsets=OFF), dict(N=1 << 22, groups=512, offsets=OFF)):
        assert call(**bad) == UNSUPPORTED, bad
    for empty in (dict(T=0), dict(N=0)):  # nothing to do, nothing touched
        assert call(**empty) == ozk.OZK_OK


def test_activations():
    for bad in (-1, 3):
        assert gated(act=bad) == INVALID


@pytest.mark.parametrize("name", ["gemv.cu", "gated_grad.cu", "activation.cuh"])
def test_loads_stay_behind_the_wait_for_the_kernel_before(name):
    """As for the other kernels: no read through the non-coherent path, none that may move over the wait."""
    text = open(os.path.join(ozk_build.CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    assert "__ldg" not in text and "__restrict__" not in text
    assert not re.search(r"\bld\.global[.\w:]*\.nc\b", text)
    for m in re.finditer(r"\basm( volatile)?\s*\((.*?)\);", text, re.S):
        assert m.group(1) or not re.search(r"\"[^\"]*\bld\.", m.group(2)), m.group(2)
