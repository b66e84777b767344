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
