"""The kernels around the ordered selections start while the kernel before them still runs, as those do: they wait
before all else, read nothing by the read-only path, and cache-hinted loads are volatile."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ordered_merge_gb300", "csrc")
FILES = ["beam_kernels.cuh", "embed_kernels.cuh", "expert_kernels.cuh"]


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", text), flags=re.S)


def test_no_other_headers_launch_early():
    early = {os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cuh")) if "wait_for_stream();" in _code(os.path.basename(p))}
    assert early == set(FILES)


@pytest.mark.parametrize("name", FILES)
def test_kernels_keep_to_the_rules(name):
    code = _code(name)
    assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__|__ldc[gs]\b|__ldca\b", code)
    for asm in re.findall(r"asm\b[^;]*?\"ld\.global[^\"]*\"", code):
        assert asm.startswith("asm volatile")
    kernels = re.findall(r"__global__[^{;]*?\b(\w+_kernel)\s*\([^{;]*\)\s*\{\s*([^;]*);", code)
    assert len(kernels) == len(re.findall(r"\b__global__\b", code)) > 0
    for kernel, first in kernels:
        assert first.strip() == "wait_for_stream()", kernel
