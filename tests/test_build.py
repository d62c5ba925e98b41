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
    front = b.front_path
    monkeypatch.setattr(b, "front_path", lambda: str(tmp_path / os.path.basename(front())))
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


def test_a_front_end_of_another_torch_is_not_loaded(compiled, monkeypatch):
    torch = pytest.importorskip("torch")
    from gqa_prefix_suffix_b200 import binding as bd
    b.build()
    here = b.front_path()
    assert os.path.exists(here)
    monkeypatch.setattr(bd, "_front", None)
    monkeypatch.setattr(bd, "lib", lambda: None)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert b.front_path() != here
    with pytest.raises(RuntimeError, match="9.9.9.*missing"):
        bd._load_front()
    assert not b._fresh(b.front_path(), [])


def test_a_front_end_of_another_interpreter_is_not_loaded(monkeypatch):
    pytest.importorskip("torch")
    here = b.front_path()
    monkeypatch.setattr(b.sysconfig, "get_config_var", lambda name: "cpython-399")
    assert b.front_path() != here
