"""What build() does where a part cannot be built; no GPU needed."""
import os

import pytest

from collective_communication_gb300 import build


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The CPython module's target in an empty folder, and no Python headers; the library as it is."""
    build.build()
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    return tmp_path


def test_library_is_built_without_python_headers(elsewhere, capsys):
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert "no Python.h" in capsys.readouterr().err
    assert os.listdir(elsewhere) == []


def test_module_of_another_source_does_not_stay(elsewhere):
    stale = elsewhere / "_operands.so"
    stale.write_bytes(b"")
    os.utime(stale, (0, 0))
    build.build()
    assert not stale.exists()
