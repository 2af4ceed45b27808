"""Rules of the low-precision kernels that only their source shows."""
import os
import re

import pytest

from fp64_gemm_emulation_exponent_gb300 import build as ozk_build


def statements(name):
    """The asm statements of a kernel source, comments taken out: (volatile or not, text)."""
    text = open(os.path.join(ozk_build.CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    return text, [(m.group(1) is not None, m.group(2)) for m in re.finditer(r"\basm( volatile)?\s*\((.*?)\);", text, re.S)]


@pytest.mark.parametrize("name", ["mx4_quantize.cu", "products.cu", "tc_ptx.cuh"])
def test_loads_stay_behind_the_wait_for_the_kernel_before(name):
    """The kernels may start while the one before them still writes: a read through the non-coherent path, or one that
    the compiler may move over the wait, could see what was there before."""
    text, asms = statements(name)
    assert "__ldg" not in text
    assert not re.search(r"\bld\.global[.\w:]*\.nc\b", text)
    for volatile, body in asms:
        assert volatile or not re.search(r"\"[^\"]*\bld\.", body), body
