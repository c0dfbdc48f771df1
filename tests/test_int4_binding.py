"""The 4-bit cache's binding on a host without CUDA."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_on_a_torch_without_cuda():
    """A torch that was built without CUDA lacks the names behind the fast device and stream queries."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from paged_kv_cache_379_b200 import ops
cache = ops.new_int4_cache(2, 16, 1, 64, device="cpu")
try:
    ops.dequantize_blocks_int4(cache, cache, torch.zeros(1, dtype=torch.int32), 64)
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise AssertionError("a CPU tensor was taken")
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
