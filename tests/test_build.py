"""The build: what it needs, and when it builds again."""
import importlib.util
import os

import pytest

from sparse_voxel_grid_leaf_gb300 import _build


@pytest.fixture
def built():
    _build.build()


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """The commands a build would run, each writing an empty file in place of its output."""
    seen = []

    def run(cmd, **kw):
        seen.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

        class Done:
            returncode, stderr = 0, ""
        return Done

    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libtb.so"))
    monkeypatch.setattr(_build, "SEQ", str(tmp_path / "_seq.so"))
    monkeypatch.setattr(_build, "SEQ_OBJ", str(tmp_path / "tb_seq_py.o"), raising=False)
    return seen


def compiled(commands):
    return [os.path.basename(c[c.index("-c") + 1]) for c in commands if "-c" in c]


def without_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_the_library_needs_no_torch(built, commands, monkeypatch, capsys):
    """Without torch libtb.so is built, and the missing entry points are said."""
    without_torch(monkeypatch)
    lib = _build.build()
    assert os.path.exists(lib) and not os.path.exists(_build.SEQ)
    assert sorted(compiled(commands)) == sorted(_build.SOURCES)
    assert "_seq.so" in capsys.readouterr().err


def test_a_second_build_does_nothing(built, commands):
    _build.build()
    first = len(commands)
    assert "tb_seq_py.cpp" in compiled(commands) and first == len(_build.SOURCES) + 3
    _build.build()
    assert len(commands) == first


def test_another_torch_is_another_build(built, commands, monkeypatch, tmp_path):
    """The entry points link torch's C++ ABI: another version, or another place, builds and links them again."""
    _build.build()
    other = tmp_path / "torch"
    other.mkdir()
    root = os.path.dirname(importlib.util.find_spec("torch").origin)
    with open(os.path.join(root, "version.py")) as f:
        (other / "version.py").write_text(f.read())
    find = importlib.util.find_spec

    class Spec:
        origin = str(other / "__init__.py")

    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: Spec if name == "torch" else find(name, *a))
    for change in (None, "__version__ = '99.0'\n"):
        if change:
            (other / "version.py").write_text(change)
        del commands[:]
        _build.build()
        assert compiled(commands) == ["tb_seq_py.cpp"] and len(commands) == 2
        del commands[:]
        _build.build()
        assert not commands
