"""The grouped linear operators' binding on the host: what it needs of torch, and its refusals."""
import os
import subprocess
import sys

import pytest

import sparse_mixture_experts_26_b200 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_package_imports_without_torchs_private_cuda_functions():
    """As in a build of torch without CUDA, where torch._C has none of them."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import sparse_mixture_experts_26_b200 as moe
x = torch.zeros(6, 16)
try:
    moe.moe_checkpoint_save(x, *moe.alloc_checkpoint(6, 16, device="cpu"))
except ValueError as e:
    assert "CUDA" in str(e)
    print("refused")
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0, run.stderr
    assert run.stdout.strip() == "refused"


@pytest.mark.parametrize("n,supported", [(1 << 30, True), ((1 << 30) + 8, False),
                                         ((1 << 31) - 1032, False), ((1 << 31) - 8, False)])
def test_row_lengths_near_2_to_the_31_are_refused(n, supported):
    """Rounded up to a tile or a checkpoint block they would leave 32 bits, and the rows behind the
    first would lie elsewhere.  Nothing is launched: too little workspace, or refused."""
    P, BF16, WORKSPACE, UNSUPPORTED = 1 << 20, 1, 3, 2
    lib = moe._lib
    for K, N in ((8, n), (n, 8)):
        assert (lib.moe_grouped_linear_workspace_bytes(2, K, N, 1, BF16) > 0) == supported
        assert (lib.moe_grouped_linear_backward_workspace_bytes(2, K, N, 1, BF16) > 0) == supported
        code = lib.moe_grouped_linear(P, None, P, None, None, 2, K, N, 1, 0, BF16, BF16, P, P, 0,
                                      None)
        assert code == (WORKSPACE if supported else UNSUPPORTED)
    if not supported:
        assert lib.moe_checkpoint_save(P, 2, n, BF16, P, P, None) == UNSUPPORTED
        assert lib.moe_checkpoint_restore(P, P, 2, n, 0, BF16, P, None) == UNSUPPORTED
