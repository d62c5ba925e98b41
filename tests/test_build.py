"""What the build compiles, with the compilers replaced by fakes."""
import os
import sys

import pytest

from gqa_prefix_suffix_b200 import build as b


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """The outputs that a build in an empty folder asked for, in order."""
    out = []

    def run(cmd, check):
        assert check
        path = cmd[cmd.index("-o") + 1]
        open(path, "w").close()
        out.append(os.path.basename(path).split(".tmp")[0])
    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "LIB", str(tmp_path / os.path.basename(b.LIB)))
    monkeypatch.setattr(b, "FRONT", str(tmp_path / os.path.basename(b.FRONT)))
    return out


def test_the_library_needs_no_torch(compiled, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)        # as if it were not installed
    assert b.build() == b.LIB
    assert compiled == ["libdm05_suffix_attn.so"] and os.path.exists(b.LIB)
    assert "torch" in capsys.readouterr().err              # says what was left out


def test_the_library_needs_no_python_headers(compiled, monkeypatch, capsys, tmp_path):
    import sysconfig
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    assert b.build() == b.LIB
    assert compiled == ["libdm05_suffix_attn.so"]
    assert "Python.h" in capsys.readouterr().err


def test_both_are_built_where_both_can_be(compiled):
    pytest.importorskip("torch")
    b.build()
    assert compiled[0] == "libdm05_suffix_attn.so" and len(compiled) == 2
    assert compiled[1].startswith("_torch_front")
    b.build()                                              # nothing is stale
    assert len(compiled) == 2
    b.build(force=True)
    assert len(compiled) == 4
