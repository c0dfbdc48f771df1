"""Which kernels may let the next one of the stream start before they end: none whose
results later kernels read ahead of their own wait (queries, new rows, lengths, tables).
Read from the sources: a race of this kind is not provoked on a GPU."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_379_b200", "csrc")


def _bodies():
    """Kernel name -> source text from its __global__ to the next one's (or the file's end)."""
    out = {}
    for name in os.listdir(CSRC):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        starts = [m.start() for m in re.finditer(r"__global__", text)]
        for a, b in zip(starts, starts[1:] + [len(text)]):
            head = text[a:text.index("{", a)]
            kernel = re.search(r"(\w+_kernel)\s*\(", head)
            if kernel:
                out[kernel.group(1)] = text[a:b]
    return out


@pytest.mark.parametrize("kernel", ["prepare_batch_kernel", "fill_tokens_kernel", "release_blocks_kernel", "row_kernel",
                                    "dequantize_blocks_int4_kernel", "decode_int4_kernel"])
def test_writers_of_early_read_arrays_hold_the_next_kernel_back(kernel):
    body = _bodies()[kernel]
    assert "pdl_wait()" in body and "pdl_launch_dependents()" not in body


@pytest.mark.parametrize("kernel", ["store_int4_kernel", "reshape_and_cache_kernel", "reshape_and_cache_fp8_kernel",
                                    "copy_blocks_kernel", "swap_blocks_kernel", "append_kv_kernel",
                                    "append_kv_cow_kernel", "lse_reduce_kernel"])
def test_the_others_start_the_next_one_after_their_own_wait(kernel):
    """A kernel that let the next one start ahead of its own wait would let it past the kernel before, too."""
    body = _bodies()[kernel]
    assert 0 <= body.index("pdl_wait()") < body.index("pdl_launch_dependents()")
