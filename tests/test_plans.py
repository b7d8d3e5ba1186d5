"""The host's choices of kernel, tile and split (csrc/norm_fp4_plan.cuh), evaluated
without a GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """Plans of a list of lines: a list of lists of integers."""
    nvcc = os.environ.get("NVCC", "nvcc")
    if shutil.which(nvcc) is None:
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("plans") / "print_plans")
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "--expt-relaxed-constexpr", "-I",
                    os.path.join(ROOT, "fp8_block_scaled_11_b200", "csrc"),
                    os.path.join(ROOT, "tests", "plans", "print_plans.cu"), "-o", exe], check=True)

    def run(lines):
        out = subprocess.run([exe], input="\n".join(lines), check=True, capture_output=True, text=True).stdout
        return [[int(v) for v in line.split()] for line in out.splitlines()]
    return run


SIZES = [(m, n, k) for m in (1, 16, 33, 128, 129, 256, 512, 777, 1024, 4096, 16640)
         for n in (1, 1000, 5120, 32000) for k in (32, 256, 2080, 8192, 70016)]


def test_product_without_pairs(plans):
    """Where CTA pairs cannot run, every product has a plan on single CTAs, and one that needed no pairs keeps its own."""
    with_pairs = plans([f"fp4 {m} {n} {k} 148 1" for m, n, k in SIZES])
    without = plans([f"fp4 {m} {n} {k} 148 0" for m, n, k in SIZES])
    assert any(p[0] for p in with_pairs)
    for (m, n, k), p, s in zip(SIZES, with_pairs, without):
        pair, bn, tiles_m, tiles_n, parts, splits, ws = s
        assert not pair and bn in (16, 32, 64, 128) and parts in (1, 2, 4, 8) and splits >= 1
        assert tiles_m == -(-m // bn) and tiles_n == -(-n // 128)
        if not p[0]:
            assert p == s
        else:
            assert p[1] == 256 and p[5] == 1 and p[6] == 0       # the size of no workspace is what a caller is told
