"""The instruction descriptor of tcgen05.mma kind::mxf4.block_scale
(csrc/ptx_fp4.cuh), evaluated on the host, field by field against the PTX ISA's
table for that kind: bits 0-1 reserved, 2 sparsity (0), 3 reserved, 4-5 the B
scale-factor id (0 or 2), 6 reserved, 7-9 / 10-11 the A / B format (1 = E2M1),
12 reserved, 13 / 14 negate, 15 / 16 major (0 = K), 17-22 N >> 3, 23 the scale
type (1 = UE8M0), 24-26 reserved, 27-28 M >> 7, 29-30 the A scale-factor id, 31
the K size (0 = 64)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def field(v, lo, width):
    return (v >> lo) & ((1 << width) - 1)


def test_instruction_descriptor(tmp_path):
    nvcc = os.environ.get("NVCC", "nvcc")
    if shutil.which(nvcc) is None:
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "print_descriptors_fp4")
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-I",
                    os.path.join(ROOT, "fp8_block_scaled_11_b200", "csrc"),
                    os.path.join(ROOT, "tests", "descriptors", "print_descriptors_fp4.cu"), "-o", exe], check=True)
    lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines()
    assert len(lines) == 12
    for line in lines:
        M, N, sf_id, v = (int(t) for t in line.split()[1:])
        assert field(v, 0, 4) == 0 and field(v, 6, 1) == 0 and field(v, 12, 5) == 0 and field(v, 24, 3) == 0
        assert field(v, 4, 2) == sf_id and field(v, 29, 2) == sf_id
        assert field(v, 7, 3) == 1 and field(v, 10, 2) == 1
        assert field(v, 17, 6) == N >> 3 and field(v, 27, 2) == M >> 7
        assert field(v, 23, 1) == 1 and field(v, 31, 1) == 0
