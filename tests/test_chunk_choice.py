"""The bound on contexts of a chunk attention call: its refusals and its place in the
C structure (no GPU needed; the fake pointers are never dereferenced)."""

import ctypes
import inspect
import os
import re

import pytest

from test_chunk_refusals import WS, chunk, ref, scales
from test_serving_refusals import FAKE, INVALID, L, cache  # noqa: F401


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("bad", [-1, -2 ** 31])
def test_negative_bounds_are_refused(L, bad, q8):  # noqa: F811
    s = ref(scales()) if q8 else None
    assert L.bsa_chunk_attention(ref(chunk(max_context=bad)), ref(cache()), s, FAKE, WS, None) == INVALID


def test_the_header_and_the_binding_name_the_same_fields():
    from block_sparse_flashattention_bsa_gb300._binding import _ChunkArgs
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "bsa.h")) as f:
        body = re.search(r"typedef struct \{([^}]*)\} bsa_chunk_args;", f.read()).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n.strip(" *\n") for d in body.split(";") if d.strip() for n in re.sub(r"^\s*(const )?(\w+)\s", "", d).split(",")]
    assert names == [n for n, _ in _ChunkArgs._fields_]
    assert ctypes.sizeof(_ChunkArgs) == 72


def test_the_python_call_has_no_bound_unless_given():
    from block_sparse_flashattention_bsa_gb300 import chunk_attention
    p = inspect.signature(chunk_attention).parameters
    assert p["max_context"].default == 0 and list(p)[-1] == "max_context"
