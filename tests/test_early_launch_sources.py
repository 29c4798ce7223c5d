"""Kernels that start while the kernel before them in the stream still runs: what their sources have to keep to.

Such a kernel's inputs may still be written after it has started, so the read-only data path, which wants
memory that nobody writes for as long as the kernel lives, is closed to it, and it waits before all else.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ordered_merge_gb300", "csrc")


def _code(path):
    text = open(path).read()
    return re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", text), flags=re.S)


EARLY = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")) if "wait_for_stream" in _code(p))


def test_there_are_such_kernels():
    assert EARLY == ["evict.cu", "group.cu", "route.cu"]


@pytest.mark.parametrize("name", [*EARLY, "select_common.cuh"])
def test_no_loads_by_the_read_only_path(name):
    code = _code(os.path.join(CSRC, name))
    assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", code)
    # loads with a cache hint: volatile, so that the compiler cannot lift them over the wait
    assert not re.search(r"__ldc[gs]\b|__ldca\b", code)
    for asm in re.findall(r"asm\b[^;]*?\"ld\.global[^\"]*\"", code):
        assert asm.startswith("asm volatile")


@pytest.mark.parametrize("name", EARLY)
def test_the_wait_comes_first(name):
    code = _code(os.path.join(CSRC, name))
    kernels = re.findall(r"__global__[^{;]*?\b(\w+_kernel)\s*\([^{;]*\)\s*\{\s*([^;]*);", code)
    assert len(kernels) == len(re.findall(r"\b__global__\b", code))
    for kernel, first in kernels:
        assert first.strip() == "wait_for_stream()", kernel
