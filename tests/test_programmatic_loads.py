"""Kernels that may start before the one in front of them has ended read memory
with coherent loads only (no GPU: the sources are read).

What such a kernel reads may be written by the kernel before it, during its own
lifetime.  The non-coherent path (__ldg, ld.global.nc, and what a compiler may make
of a load through a pointer declared const and __restrict__) is defined only for
memory that nobody writes while the kernel runs, and a load that promises so may be
moved in front of griddepcontrol.wait.  Cache-hinted loads are the wrappers of
ptx_load.cuh, which no compiler moves across that wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_11_b200", "csrc")
FILES = ["norm_kernels.cuh", "fp4_quant_kernels.cuh", "gemm_fp4_kernel.cuh", "gemm_fp4_pair_kernel.cuh",
         "splitk_reduce.cuh", "mx4.cuh", "ptx_fp4.cuh", "ptx_load.cuh"]


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_promises(name):
    text = source(name)
    for word in ("__ldg", "ld.global.nc", "__restrict__", "__ldcs", "__ldcg", "__ldca"):
        assert not re.search(re.escape(word) + r"\b", text), f"{name}: {word}"
    # Vec8::load is the 8-bit kernels', which are launched in stream order
    assert not re.search(r"\.load\(", text), f"{name}: Vec8::load"


def test_every_programmatic_kernel_waits_first():
    """Each of these kernels reaches the wait, by its own body or by ring_init."""
    for name in FILES:
        for body in re.split(r"__global__", source(name))[1:]:
            kernel = re.search(r"(\w+_kernel)\(", body).group(1)
            assert re.search(r"grid_begin\(\)|ring_init\(|griddepcontrol\.wait", body), kernel


def test_wrappers_are_ordered():
    """The loads' wrappers are volatile and clobber memory."""
    text = source("ptx_load.cuh")
    found = re.findall(r"asm(.{0,12})\(\s*\"ld\.global[^;]*;\"(.*?)\);", text, flags=re.S)
    assert len(found) >= 3
    for head, tail in found:
        assert "volatile" in head and '"memory"' in tail
