"""The build: the library does not need the binding, and the binding follows the installed torch."""
from __future__ import annotations

import ctypes
import os

import pytest

from gated_delta_rule_sm_gb300 import build as kbuild


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of one small source in a folder of its own."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    for name, value in dict(PKG=tmp_path, BUILD_DIR=tmp_path / "obj", LIB_PATH=tmp_path / "lib.so", OPS_PATH=tmp_path / "ops.so",
                            OPS_TORCH=tmp_path / "obj" / "torch").items():
        monkeypatch.setattr(kbuild, name, str(value), raising=False)
    monkeypatch.setattr(kbuild, "sources", lambda: [str(src)])
    return tmp_path


def test_library_is_built_without_the_binding(elsewhere, monkeypatch):
    def no_headers():
        raise RuntimeError("no torch headers")

    monkeypatch.setattr(kbuild, "_compile_ops", no_headers)
    with pytest.raises(RuntimeError, match="no torch headers"):
        kbuild.build()
    assert ctypes.CDLL(str(elsewhere / "lib.so")).one() == 1
    assert not os.path.exists(elsewhere / "ops.so")


def test_another_torch_is_another_build(monkeypatch):
    kbuild.build()
    assert kbuild.up_to_date()
    monkeypatch.setattr("torch.__version__", "0.0.0")
    assert not kbuild.up_to_date()
