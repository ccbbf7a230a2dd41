"""The build without torch, and for another torch than the last one's."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "post_weight_quantization_13_b200"


@pytest.fixture()
def build():
    import __graft_entry__
    __graft_entry__.build()
    return __graft_entry__._builder()


def test_the_library_builds_without_torch(build, monkeypatch, tmp_path, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)            # as where it is not installed
    monkeypatch.setattr(build, "EXT", str(tmp_path / "_serving.so"))
    assert build.build() == build.LIB
    assert not os.path.exists(build.EXT)
    assert "torch is not installed" in capsys.readouterr().err


def test_the_serving_module_is_built_anew_for_another_torch(build, monkeypatch):
    assert build.ext_up_to_date()
    built = []
    monkeypatch.setattr(build, "build_ext", lambda verbose: built.append(1))
    build.build()
    assert not built
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "0.0")
    build.build()
    assert built == [1]
