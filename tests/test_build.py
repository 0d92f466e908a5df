"""What build.py builds, without compiling: commands are recorded in place of run. CPU only."""
import importlib.util
import os

import pytest

from persistent_megakernel_interpreter_b200 import build


@pytest.fixture
def recorded(monkeypatch, tmp_path):
    """build.py's outputs under tmp_path; every compiler call writes its output file and is recorded."""
    done = []

    def run(cmd):
        done.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmk.so"))
    monkeypatch.setattr(build, "CALL", str(tmp_path / "_call.so"))
    monkeypatch.setattr(build, "CALL_STAMP", str(tmp_path / "_call.stamp"), raising=False)
    monkeypatch.setattr(build.subprocess, "check_call", run)
    return done


def test_the_library_is_built_without_torch(monkeypatch, recorded, capsys):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build_library() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALL)
    assert not any(build.CALL_SOURCE in cmd for cmd in recorded)
    assert "_call.so" in capsys.readouterr().err
    recorded.clear()
    build.build_library()                                    # the library is up to date: nothing is compiled
    assert not recorded


def test_another_torch_makes_the_binding_stale(monkeypatch, recorded, tmp_path):
    """Its machine code belongs to one torch, whose files may be older than it."""
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "version.py").write_text("__version__ = '1'\n")
    find = importlib.util.find_spec

    class Spec:
        submodule_search_locations = [str(torch)]
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: Spec if name == "torch" else find(name, *a))
    bindings = lambda: sum(build.CALL_SOURCE in cmd for cmd in recorded)
    build.build_library()
    assert bindings() == 1
    build.build_library()
    assert bindings() == 1
    (torch / "version.py").write_text("__version__ = '2'\n")
    os.utime(torch / "version.py", (0, 0))
    build.build_library()
    assert bindings() == 2
    build.build_library()
    assert bindings() == 2
