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
