"""Kernels that are launched while the kernel before them still runs (csrc/pdl.cuh) overlap in time with the one that
writes their operands.  Loads through the non-coherent path are for memory that nobody writes while a kernel lives,
so these kernels have none, written out or left to the compiler (const __restrict__ parameters)."""
import glob
import os
import re

import pytest

from rotated_w4a8_int8_gb300 import _build


def code(path):
    with open(path) as f:
        src = f.read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", src, flags=re.S))


def sources():
    found = [p for p in sorted(glob.glob(os.path.join(_build.CSRC, "*.cu"))) if "launch_after(" in code(p)]
    assert len(found) >= 4
    return found + [os.path.join(_build.CSRC, "epilogue.cuh"), os.path.join(_build.CSRC, "pdl.cuh")]


@pytest.mark.parametrize("path", sources(), ids=os.path.basename)
def test_no_non_coherent_loads(path):
    assert not re.findall(r"__ldg\b|ld\.global[.\w:]*\.nc\b|__restrict__", code(path))
