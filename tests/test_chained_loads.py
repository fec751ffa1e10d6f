"""Kernels of consecutive calls overlap: one starts while the kernel before it
may still write what it will read, and waits (griddepcontrol.wait) before it
reads. A read-only load (ld.global.nc: __ldg, or a const __restrict__ pointer)
is defined only for data that nobody writes while the kernel runs, and need not
stay behind the wait. So such kernels read by plain loads."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_kv_cache_ott_gb300", "csrc")
BYTE = ["ott_byte.cuh", "ott_byte.cu", "ott_byte_rows.cu", "ott_byte_tiles.cu", "ott_select.cuh"]
# (ott_topk.cu's bounds and ott_rope.cu's kernels are launched as ordinary kernels, behind everything before them)
CHAINED = BYTE + ["ott_chunk.cuh", "ott_chunk.cu", "ott_chunk_tiles.cu", "ott_decode.cu", "ott_flush.cu", "ott_internal.cuh"]


@pytest.mark.parametrize("name", CHAINED)
def test_no_read_only_loads(name):
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    text = re.sub(r"//[^\n]*", "", text)
    found = re.findall(r"__ldg\b|ld\.global\.nc|const [\w ]+\*\s*__restrict__", text)
    assert not found, found


def test_every_kernel_of_the_8_bit_cache_waits():
    """(The release of blocks is launched as an ordinary kernel, behind everything before it.)"""
    kernels = waits = 0
    for name in BYTE:
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        parts = re.split(r"__global__", text)[1:]
        for part in parts:
            kernel = re.search(r"\b(k_\w+)\s*\(", part).group(1)
            body = part[:part.index("\n}\n")]
            if kernel != "k_byte_release":
                kernels += 1
                waits += "griddepcontrol.wait" in body
    assert kernels == waits == 7, (kernels, waits)
