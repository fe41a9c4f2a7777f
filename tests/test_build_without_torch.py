"""The C library needs nvcc alone: where torch is missing, or the binding's caller does not compile, it is linked all
the same."""
import importlib.util
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def lib_build(monkeypatch, tmp_path):
    """build.py by its path, as a user without torch runs it, with one small source and an output folder of its own."""
    spec = importlib.util.spec_from_file_location("da_build_alone", os.path.join(ROOT, "decode_attention_output_gb300", "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.setattr(m, "LIB_DIR", str(tmp_path))
    monkeypatch.setattr(m, "SOURCES", ["oproj_gemv.cu"])
    return m


def test_without_torch(lib_build, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # `import torch` raises ImportError
    for _ in range(2):  # compiled, then found up to date
        out = lib_build.build()
        assert out == lib_build.lib_path() and os.path.exists(out)
    assert not os.path.exists(lib_build.dispatch_path())


def test_when_the_caller_does_not_compile(lib_build, monkeypatch):
    def broken(force=False):
        raise RuntimeError("g++ failed on dispatch.cpp")

    monkeypatch.setattr(lib_build, "build_dispatch", broken)
    for _ in range(2):
        with pytest.raises(RuntimeError, match="g[+][+] failed"):
            lib_build.build()
        assert os.path.exists(lib_build.lib_path())
