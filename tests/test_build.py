"""What build() promises, without a GPU."""
import os

import pytest

from sequence_long_context_zigzag_gb300 import build


@pytest.mark.parametrize("cxx", ["false", "/nonexistent/g++"])
def test_the_library_is_built_where_the_binding_cannot_be(cxx, monkeypatch, tmp_path):
    monkeypatch.setenv("CXX", cxx)
    monkeypatch.setattr(build, "binding_path", lambda: str(tmp_path / "binding.so"))
    with pytest.warns(RuntimeWarning, match="binding"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.listdir(tmp_path)
    with pytest.raises(Exception):   # who needs the binding hears of it
        build.build_binding()


def test_the_library_is_built_without_torch(monkeypatch):
    def absent():
        raise ModuleNotFoundError("No module named 'torch'")
    monkeypatch.setattr(build, "binding_path", absent)
    with pytest.warns(RuntimeWarning, match="torch"):
        assert build.build() == build.LIB


@pytest.mark.parametrize("changed", ["usp.h", "binding.cpp", "python"])
def test_a_binding_from_other_sources_is_not_loaded(changed, monkeypatch, tmp_path):
    """The module's file name changes with what it is built from, so that one from another header, source or
    interpreter is never taken for the present one."""
    import shutil
    import sysconfig
    now = build.binding_path()
    assert now == build.binding_path()
    if changed == "python":
        monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-x86_64-linux-gnu")
    else:
        src = os.path.join(build.INCLUDE, "usp.h") if changed == "usp.h" else build.BINDING_SRC
        copy = str(tmp_path / changed)
        shutil.copy(src, copy)
        with open(copy, "a") as f:
            f.write("\n")
        if changed == "usp.h":
            monkeypatch.setattr(build, "INCLUDE", str(tmp_path))
        else:
            monkeypatch.setattr(build, "BINDING_SRC", copy)
    assert build.binding_path() != now


def test_the_binding_is_built_from_its_present_sources(monkeypatch, tmp_path):
    """The package loads what build_binding() gives for the present sources, and builds it where there is none."""
    from sequence_long_context_zigzag_gb300 import _abi
    path, built = str(tmp_path / "binding.so"), []
    monkeypatch.setattr(build, "binding_path", lambda: path)
    monkeypatch.setattr(build, "_build_binding", lambda p: built.append(p) or open(p, "w").close())
    monkeypatch.setattr(_abi, "_binding", None)
    with pytest.raises(ImportError):    # an empty file is no module
        _abi.binding()
    assert built == [path]
