"""The C library is built whether or not the Python binding can be."""
import os
import sys

import pytest

from moe_layer_amd import build as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not found")


@pytest.fixture
def small(tmp_path, monkeypatch):
    """build.py on a source tree of one empty unit, with a binding that would compile."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "one.hip").write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    (csrc / "binding.cpp").write_text("int two() { return 2; }\n")
    monkeypatch.setattr(B, "CSRC", str(csrc))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_binding.so"))
    return tmp_path


def test_library_and_binding(small):
    assert B.build(verbose=False) == str(small / "lib.so")
    assert (small / "lib.so").exists() and (small / "_binding.so").exists()


def test_library_without_torch(small, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)        # as if it were not installed
    assert B.build(verbose=False) == str(small / "lib.so")
    assert (small / "lib.so").exists() and not (small / "_binding.so").exists()


def test_library_stands_when_the_binding_fails(small):
    (small / "csrc" / "binding.cpp").write_text("no C++\n")
    with pytest.raises(RuntimeError, match="binding"):
        B.build(verbose=False)
    assert (small / "lib.so").exists() and not (small / "_binding.so").exists()
