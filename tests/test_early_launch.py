"""Kernels that are launched while the kernel before them still runs see what it wrote
after their wait, by ordinary loads.  Read-only loads are for memory that nobody writes
during the whole kernel, so no file with such a launch may use them (no GPU needed)."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_sparse_flashattention_bsa_gb300", "csrc")


def code(path):
    with open(path) as f:
        s = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", s, flags=re.S)


EARLY = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")) if "launch_after(" in code(p))


def test_there_are_such_files():
    assert {"bsa_cache.cu", "bsa_chunk.cu", "bsa_decode.cu", "bsa_read.cu", "bsa_rope.cu", "bsa_tree.cu"} <= set(EARLY)


@pytest.mark.parametrize("name", EARLY + ["bsa_chunk.cuh", "bsa_q8.cuh", "bsa_ptx.cuh"])
def test_no_read_only_loads(name):
    s = code(os.path.join(CSRC, name))
    # __restrict__ const pointers are loaded that way too, where the compiler sees fit
    for word in ("__ldg", r"ld\.global\S*\.nc", "__restrict__", "tex1D"):
        assert not re.search(word, s), word


@pytest.mark.parametrize("name", EARLY)
def test_every_kernel_waits(name):
    """Each kernel of such a file waits for the one before it."""
    s = code(os.path.join(CSRC, name))
    bodies = re.split(r"__global__", s)[1:]
    kernels = [b for b in bodies if "griddep_launch_dependents()" in b]
    assert kernels and all("griddep_wait()" in b for b in kernels)
