"""The grouped linear operators' binding on the host: what it needs of torch, and its refusals."""
import os
import subprocess
import sys

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
