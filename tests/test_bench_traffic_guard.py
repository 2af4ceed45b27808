"""The committed DRAM traffic of the residue GEMM counts in a bench line only while every file of the kernel is the one
it was measured on."""
import os
import re

import bench
from fp64_gemm_emulation_exponent_gb300 import build as ozk_build


def sources(name, seen):
    """The kernel's file and all it includes from beside it."""
    if name in seen or not os.path.exists(os.path.join(ozk_build.CSRC, name)):
        return seen
    seen.add(name)
    for other in re.findall(r'#include "([^"]+)"', open(os.path.join(ozk_build.CSRC, name)).read()):
        sources(other, seen)
    return seen


def test_the_hash_covers_every_file_of_the_kernel():
    assert sources("residue_gemm.cu", set()) == set(bench.KERNEL_SOURCES)


def test_the_committed_traffic_belongs_to_the_kernel():
    assert bench.committed_traffic("square4096_normal/n14") > 10 ** 9


def test_another_file_voids_it(monkeypatch, tmp_path):
    for name in bench.KERNEL_SOURCES:
        with monkeypatch.context() as m:
            root = tmp_path / name
            csrc = root / "fp64_gemm_emulation_exponent_gb300" / "csrc"
            csrc.mkdir(parents=True)
            for f in bench.KERNEL_SOURCES:
                text = open(os.path.join(ozk_build.CSRC, f)).read()
                (csrc / f).write_text(text + "\n" if f == name else text)
            m.setattr(bench, "ROOT", str(root))
            assert bench.committed_traffic("square4096_normal/n14") is None
