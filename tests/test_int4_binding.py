"""The 4-bit cache's and the batch preparation's calls on a host without a GPU."""

import ctypes
import os
import subprocess
import sys

from paged_kv_cache_379_b200 import _lib

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


def test_prepare_batch_refuses_shifted_overlaps():
    P = ctypes.c_void_p
    at = dict(bt=0x10000, ctx=0x20000, new=0x30000, free=0x40000, nf=0x50000, sl=0x60000, qs=0x70000, ids=None, pos=None,
              slots=None, nfo=0x80000, status=0x90000)

    def call(**kw):
        ptrs = [v and P(v) for v in dict(at, **kw).values()]
        return _lib.load().pa_prepare_batch(*ptrs, 4, 8, 16, 100, 16, 100, None)

    for kw in (dict(sl=0x20004), dict(sl=0x1FFFC), dict(sl=0x3000C), dict(sl=0x2FFF4), dict(qs=0x20000), dict(qs=0x2FFF0),
               dict(qs=0x3000C)):
        assert call(**kw) == -2, kw
