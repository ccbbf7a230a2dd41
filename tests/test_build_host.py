"""The build without torch, and for another torch than the last one's."""
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


def _python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_every_name_imports_with_torch_and_the_librarys_without(build):
    r = _python(f"from {PACKAGE} import *\nassert callable(linear_int8) and callable(solve_layer)")
    assert r.returncode == 0, r.stderr
    r = _python(f"import sys\nsys.modules['torch'] = None\nfrom {PACKAGE} import *\n"
                "assert gptq_abi_version() and callable(gptq_validate_config) and 'linear_int8' not in globals()")
    assert r.returncode == 0, r.stderr
