"""Workspaces are sized for the device that they are allocated on, which need not
be the current one (no GPU: the extension module is a fake)."""
import types

import pytest
import torch

from fp8_block_scaled_11_b200 import build, ops


@pytest.fixture
def asked(monkeypatch):
    """The calls that ask for sizes: (name, arguments)."""
    calls = []

    def answer(name, size):
        return lambda *args: calls.append((name, args)) or size
    monkeypatch.setattr(ops, "_native", types.SimpleNamespace(
        product_workspace=answer("product", 0), norm_backward_workspace=answer("backward", 4096)))
    return calls


@pytest.mark.parametrize("device,index", [("cuda:1", 1), (torch.device("cuda", 3), 3), ("cuda", -1), ("cpu", -1), (2, 2),
                                          (None, -1)])
def test_product(asked, device, index):
    assert ops.fp4_scaled_gemm_workspace(16, 130, 131072, device) is None
    assert asked == [("product", (16, 130, 131072, index))]


def test_backward(asked, monkeypatch):
    made = []
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: made.append((shape, dtype, device)))
    dev = torch.device("cuda", 1)
    ops.rmsnorm_backward_workspace(types.SimpleNamespace(shape=(333, 1040), device=dev))
    assert asked == [("backward", (333, 1040, 1))]
    assert made == [((4096,), torch.uint8, dev)]


def test_sizes_of_the_module():
    """-1: whatever device is current; the C entry points' sizes."""
    build.build()
    native, lib = ops._load_native(), ops.lib()
    for m, n, k in ((1, 5120, 8192), (16, 130, 131072), (0, 1, 32)):
        assert native.product_workspace(m, n, k, -1) == lib.fp4_scaled_gemm_workspace_size(m, n, k)
    for rows, cols in ((1, 16), (333, 1040), (5, 16400), (0, 16)):
        assert native.norm_backward_workspace(rows, cols, -1) == lib.fp8bs_rmsnorm_backward_workspace_size(rows, cols)
