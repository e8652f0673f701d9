"""The package on a PyTorch built without CUDA: it imports, and what needs no GPU
works."""
import subprocess
import sys

from conftest import ROOT

SCRIPT = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
torch.cuda.is_available = lambda: False
import block_sparse_masked_mask_gb300 as pkg
from block_sparse_masked_mask_gb300 import ulysses, workloads
w = workloads.random_workload(1, "shared_prefix", [40, 15], num_heads=2, head_dim=32)
assert w.total_tokens == 55
try:
    pkg.attn_rope(torch.zeros(3, 1, 32), None, None)
except pkg.AttnError:
    print("imported")
"""


def test_imports_without_cuda_bindings():
    run = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "imported", run.stderr
