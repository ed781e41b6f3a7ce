"""The build script: the C library does not depend on the Python binding's parts."""
import os

import pytest

from draft_sampling_verification_02_amd import build


def test_the_c_library_is_built_where_the_binding_module_cannot_be(tmp_path, monkeypatch):
    # one source stands for all; no host compiler for the marshalling module
    monkeypatch.setattr(build, "SOURCES", ["schedule.cpp"])
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "m.so"))
    monkeypatch.setattr(build, "CXX", str(tmp_path / "no-such-compiler"))
    with pytest.raises((RuntimeError, OSError), match="no-such-compiler"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.MARSHAL)
