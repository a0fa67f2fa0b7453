"""The build without a binding, and the binding under another PyTorch."""
import os
import subprocess
import sys

import pytest

from bit_routed_expert_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A build of one small source, into a folder of its own, without bind.cpp."""
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "one.hip").write_text('extern "C" int one() { return 1; }\n')
    for name, path in (("CSRC", "csrc"), ("BUILD_DIR", "_build"), ("LIB", "lib.so"), ("BIND", "_bind.so")):
        monkeypatch.setattr(build, name, str(tmp_path / path))
    return tmp_path


def test_the_library_is_linked_where_the_binding_fails(small):
    with pytest.raises(RuntimeError, match="bind.cpp"):
        build.build()
    assert (small / "lib.so").exists() and not (small / "_bind.so").exists()


def test_the_library_is_built_without_pytorch(small, monkeypatch):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build() == str(small / "lib.so")
    assert (small / "lib.so").exists()


def test_the_binding_refuses_another_pytorch():
    code = ("import torch, bit_routed_expert_amd as moe\n"
            "torch.__version__ = '0.0'\n"
            "try:\n    moe._ext()\nexcept ImportError as e:\n    print('refused', e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.stdout.startswith("refused") and "0.0" in r.stdout, r.stdout + r.stderr
