"""The C library does not need what only the Python binding's compiled part is built with (g++, torch).  CPU only."""
import importlib.metadata
import os

import pytest

from decode_packed_bit_b200 import build as lb_build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The library as it is; the compiled part, an older one, in a place of its own."""
    lb_build.build()
    monkeypatch.setattr(lb_build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(lb_build, "MARSHAL_STAMP", str(tmp_path / ".marshal.sha1"))
    for name in (lb_build.MARSHAL, lb_build.MARSHAL_STAMP):
        with open(name, "w") as f:
            f.write("older")
    return monkeypatch


def left_out():
    with pytest.warns(UserWarning, match="_marshal.so.*decode-side") as w:
        assert lb_build.build() == lb_build.LIB
    assert os.path.exists(lb_build.LIB)
    assert not os.path.exists(lb_build.MARSHAL) and not os.path.exists(lb_build.MARSHAL_STAMP)  # nothing stale stays
    return str(w[0].message)


def test_without_a_compiler(elsewhere):
    elsewhere.setenv("CXX", "/nowhere/g++")
    assert "FileNotFoundError" in left_out()


def test_without_torch(elsewhere):
    def version(name):
        raise importlib.metadata.PackageNotFoundError(name)
    elsewhere.setattr(importlib.metadata, "version", version)
    assert "PackageNotFoundError" in left_out()


def test_with_a_compiler_that_fails(elsewhere):
    elsewhere.setenv("CXX", "false")
    assert "g++ failed" in left_out()


def test_the_library_first(elsewhere):
    """Also when it has to be built: the compiled part's failure is met after it."""
    order = []
    elsewhere.setattr(lb_build, "_build_library", lambda *a: order.append("library") or lb_build.LIB)

    def fail(force=False):
        order.append("compiled part")
        raise RuntimeError("no")
    elsewhere.setattr(lb_build, "build_marshal", fail)
    left_out()
    assert order == ["library", "compiled part"]


def test_an_unknown_fault_is_not_a_warning(elsewhere):
    elsewhere.setattr(lb_build, "build_marshal", lambda force=False: 1 // 0)
    with pytest.raises(ZeroDivisionError):
        lb_build.build()
