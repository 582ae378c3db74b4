"""CPU-only: what the build compiles, with torch and without."""
import os
import sys

import pytest

from tiled_tensor_core_03_gb300 import _build


def _commands(monkeypatch):
    ran = []
    monkeypatch.setattr(_build.subprocess, "run", lambda cmd, check: ran.append(cmd))
    _build.build()
    return ran


def test_build_compiles_the_library_and_the_extension(monkeypatch):
    pytest.importorskip("torch")
    targets = {c[c.index("-o") + 1] for c in _commands(monkeypatch)}
    assert targets == {_build.LIB, _build.BINDING}


def test_build_without_torch_compiles_the_library(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    ran = _commands(monkeypatch)
    assert [c[c.index("-o") + 1] for c in ran] == [_build.LIB]
    monkeypatch.setattr(_build, "BINDING", os.path.join(_build.PKG, "not_there.so"))
    assert _build.needs_build() == _build._stale(_build.LIB, _build.DEPS)
