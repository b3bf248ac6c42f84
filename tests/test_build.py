"""What build() makes and when, with the compilers stood in for (no nvcc, no GPU)."""

import importlib
import os
import subprocess

import pytest


@pytest.fixture
def B(tmp_path, monkeypatch):
    """The build module over an empty tree; `made` lists what was compiled and linked."""
    m = importlib.import_module("block_sparse_flashattention_bsa_gb300.build")
    made = []
    for name, f in (("LIB", "libbsa.so"), ("BINDING", "_bsa_torch.so"), ("BUILD", "_build")):
        monkeypatch.setattr(m, name, str(tmp_path / f))

    def compiled(src, verbose):
        made.append(src)
        return str(tmp_path / (src + ".o"))

    def link(cmd, out):
        made.append(os.path.basename(out))
        open(out, "w").close()

    def run(cmd, **kw):
        assert m.BINDING_SOURCE in " ".join(cmd)
        made.append(m.BINDING_SOURCE)
        return subprocess.CompletedProcess(cmd, m.binding_rc, "", "no Python.h")

    monkeypatch.setattr(m, "_compile", compiled)
    monkeypatch.setattr(m, "_link", link)
    monkeypatch.setattr(m.subprocess, "run", run)
    monkeypatch.setattr(m, "nvcc", lambda: "/cuda/bin/nvcc")
    monkeypatch.setattr(m, "binding_rc", 0, raising=False)
    m.made = made
    yield m
    del m.made


def test_everything_once(B):
    assert B.build() == B.LIB
    assert sorted(B.made) == sorted(B.SOURCES + ["bsa_torch.cpp", "libbsa.so", "_bsa_torch.so"])
    B.made.clear()
    assert B.build() == B.LIB and B.made == []


def test_the_library_does_not_need_the_binding(B, monkeypatch):
    """Where the binding does not compile (no headers of torch or Python), the C
    library is linked all the same, the failure is raised, and only the binding
    is tried again."""
    monkeypatch.setattr(B, "binding_rc", 1)
    with pytest.raises(RuntimeError, match="bsa_torch.cpp"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)
    B.made.clear()
    monkeypatch.setattr(B, "binding_rc", 0)
    assert B.build() == B.LIB and B.made == ["bsa_torch.cpp", "_bsa_torch.so"]


def test_the_library_does_not_need_torch(B, monkeypatch):
    """Without torch there is nobody to bind to: the C library alone."""
    monkeypatch.setitem(B.sys.modules, "torch", None)  # import torch raises ImportError
    assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING) and "bsa_torch.cpp" not in B.made


@pytest.mark.parametrize("change", ["torch", "python", "no record"])
def test_the_binding_follows_torch_and_python(B, monkeypatch, change):
    """The binding is compiled against one torch and one Python: with another of
    either it is built again, and the library is not."""
    import torch
    B.build()
    B.made.clear()
    if change == "torch":
        monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    elif change == "python":
        monkeypatch.setattr(B.sys, "version", "3.99.0 " + B.sys.version)
    else:
        os.remove(os.path.join(B.BUILD, B.BINDING_RECORD))
    assert B.build() == B.LIB and B.made == ["bsa_torch.cpp", "_bsa_torch.so"]
    B.made.clear()
    assert B.build() == B.LIB and B.made == []


def test_a_binding_that_failed_is_not_taken_for_the_new_one(B, monkeypatch):
    import torch
    B.build()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    monkeypatch.setattr(B, "binding_rc", 1)
    for _ in range(2):
        with pytest.raises(RuntimeError, match="bsa_torch.cpp"):
            B.build()
