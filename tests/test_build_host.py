"""What the build takes for up to date, and for whom."""
import importlib.machinery
import importlib.util
import os
import subprocess
import sys
import sysconfig

import pytest

from tiled_staged_matmul_gb300.csrc import build as tsm_build


@pytest.fixture(scope="module", autouse=True)
def built():
    tsm_build.build()


def another_python(monkeypatch, tmp_path):
    own = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: ".cpython-399.so" if name == "EXT_SUFFIX" else own(name))


def another_torch(monkeypatch, tmp_path):
    (tmp_path / "__init__.py").write_text("")
    (tmp_path / "version.py").write_text("__version__ = '99.0'\n")
    spec = importlib.machinery.ModuleSpec("torch", None, origin=str(tmp_path / "__init__.py"))
    own = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else own(name, *a))


@pytest.mark.parametrize("change", [another_python, another_torch])
def test_an_extension_module_for_another_torch_or_python(monkeypatch, tmp_path, change):
    """It is built again, and until then refused instead of loaded."""
    from tiled_staged_matmul_gb300 import binding
    assert tsm_build.up_to_date()
    change(monkeypatch, tmp_path)
    assert not tsm_build.up_to_date()
    monkeypatch.setattr(binding, "_calls", None)
    with pytest.raises(ImportError, match="another torch or Python"):
        binding._load_calls()


def no_torch(monkeypatch, tmp_path):
    monkeypatch.setitem(sys.modules, "torch", None)


def a_folder_of_its_name(monkeypatch, tmp_path):
    spec = importlib.machinery.ModuleSpec("torch", None, origin=None, is_package=True)
    own = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else own(name, *a))


@pytest.mark.parametrize("missing", [no_torch, a_folder_of_its_name])
def test_the_library_where_there_is_no_torch(monkeypatch, tmp_path, missing):
    """The C ABI needs none; the extension module is left out."""
    missing(monkeypatch, tmp_path)
    monkeypatch.setattr(tsm_build, "BUILD_DIR", str(tmp_path))
    for name in ("LIB_PATH", "CALLS_PATH", "CALLS_STAMP", "PTXAS_LOG"):
        if hasattr(tsm_build, name):
            monkeypatch.setattr(tsm_build, name, str(tmp_path / os.path.basename(getattr(tsm_build, name))))
    # (Empty units in place of the library's.)
    monkeypatch.setattr(tsm_build, "_compile", lambda src, obj, verbose, flags: subprocess.run(
        ["g++", "-x", "c++", "-c", os.devnull, "-fPIC", "-o", obj], check=True) and "")
    tsm_build.build()
    assert os.path.exists(tsm_build.LIB_PATH) and not os.path.exists(tsm_build.CALLS_PATH)
    assert tsm_build.up_to_date()
