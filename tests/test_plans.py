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


# ------------------------------------------------------------------ the norm's backward pass
RING_SMEM = 222 * 1024


@pytest.mark.parametrize("elem,mats,widest", [(2, 2, 16384), (2, 3, 16384), (4, 2, 14128), (4, 3, 9424)])
def test_backward_widths(plans, elem, mats, widest):
    """Every width up to the stated one goes over the ring, no wider one does, whatever the rows."""
    cols = list(range(16, 20000, 16))
    for rows in (1, 5, 300, 20000):
        got = plans([f"back {rows} {c} {elem} {mats} 148" for c in cols])
        assert [c for c, p in zip(cols, got) if p[1] > 0] == list(range(16, widest + 1, 16))


@pytest.mark.parametrize("elem,mats", [(2, 2), (2, 3), (4, 2), (4, 3)])
def test_backward_plans_fit_their_kernels(plans, elem, mats):
    """Threads, shared memory, named barriers, partial sums and workspace of every plan are within what the kernels have."""
    at = [(r, c) for r in (1, 2, 3, 16, 17, 64, 100, 255, 256, 257, 443, 444, 2000, 16640, 100000)
          for c in [*range(16, 1100, 16), *range(1104, 17000, 208), 8192, 16384, 16400, 40000]]
    for (rows, cols), (tx, vpt, ty, slots, cluster, ctas, smem, nbytes) in zip(
            at, plans([f"back {r} {c} {elem} {mats} 148" for r, c in at])):
        if vpt == 0:
            assert 1 <= ctas <= rows and nbytes >= 4 * (ctas * cols + rows)
            continue
        eights, row = -(-cols // 8), cols * elem
        assert tx * vpt >= eights and (tx == 16 or tx % 32 == 0) and (tx * ty) % 32 == 0
        # the instantiations that there are: up to 256 threads, or up to 512 with four eights (fp32: two as well)
        assert tx * ty <= 256 or (tx * ty <= 512 and (vpt == 4 or (elem == 4 and vpt == 2)))
        assert slots >= 2 and smem <= RING_SMEM and slots * mats * ty * row + 16 * slots + 16 == smem
        assert mats * ty * row < 1 << 20                                  # bytes that one barrier counts
        if tx > 32:
            assert 1 + ty <= 16 and ty * ((tx + 127) // 128 * 4) <= 16    # a named barrier and partial sums for each row
        assert ty * cols * 4 <= slots * mats * ty * row                   # the sums of dweight take the ring's place
        if cluster:
            assert vpt in (1, 2) and tx * ty <= 256 and ctas == cluster and cluster in (1, 2, 4, 8)
        else:
            assert 1 <= ctas <= -(-rows // ty) and nbytes >= 4 * ctas * cols
