"""The library is built where the operators' Python binding cannot be."""
import os
import subprocess
import sys

import pytest

from invariant_deterministic_gemm_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def small(tmp_path, monkeypatch):
    """_build with one tiny source, its outputs in a folder of the test's."""
    src = tmp_path / "tiny.cu"
    src.write_text('extern "C" int tiny() { return 7; }\n')
    monkeypatch.setattr(_build, "sources", lambda: [str(src)])
    monkeypatch.setattr(_build, "headers", lambda: [])
    monkeypatch.setattr(_build, "OBJDIR", str(tmp_path / "obj"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libtiny.so"))
    monkeypatch.setattr(_build, "NATIVE", str(tmp_path / "native.so"))
    return tmp_path


def test_no_cxx_compiler(small, monkeypatch, capfd):
    monkeypatch.setenv("CXX", str(small / "no-such-compiler"))
    assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.NATIVE)
    assert "no-such-compiler" in capfd.readouterr().err
    assert _build.build() == _build.LIB                       # nothing to do


def test_no_python_headers(small, monkeypatch, capfd):
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(small)})
    assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.NATIVE)
    assert "Python.h" in capfd.readouterr().err


def test_a_binding_of_older_declarations_is_not_left_behind(small, monkeypatch):
    old = small / "native.so"
    old.write_text("")
    os.utime(old, (1, 1))
    monkeypatch.setenv("CXX", str(small / "no-such-compiler"))
    _build.build()
    assert not old.exists()
    old.write_text("")                                        # newer than what it declares: it stays
    _build.build(force=True)
    assert old.exists()


def test_a_call_without_the_binding_says_so():
    code = ("import sys; sys.modules['invariant_deterministic_gemm_gb300._ops_native'] = None\n"
            "import torch, invariant_deterministic_gemm_gb300 as dg\n"
            "dg.det_moe_dispatch(torch.zeros(4, 2, dtype=torch.int32), 8)\n")
    _build.build()
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode != 0 and "native binding is not built" in r.stderr
