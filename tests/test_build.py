"""When the native modules are built again (no compiler runs here)."""
import os

import pytest

from nvfp4_weight_only_flint_b200 import build as fbuild


@pytest.fixture
def runs(tmp_path, monkeypatch):
    """The extension module's build in a folder of its own, with a compiler that writes its output only."""
    made = []

    def compiler(cmd, check):
        assert check
        made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(fbuild, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(fbuild, "OBJ_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(fbuild, "MARSHAL_FOR", str(tmp_path / "_build" / "marshal.txt"), raising=False)
    monkeypatch.setattr(fbuild.subprocess, "run", compiler)
    return made


def test_extension_module_is_built_once(runs):
    for _ in range(3):
        fbuild._build_marshal(False, False)
    assert len(runs) == 1
    fbuild._build_marshal(True, False)
    assert len(runs) == 2


def test_extension_module_is_built_again_for_another_torch(runs, monkeypatch):
    import importlib.metadata
    version = importlib.metadata.version
    fbuild._build_marshal(False, False)
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "9.9" if name == "torch" else version(name))
    fbuild._build_marshal(False, False)
    assert len(runs) == 2
    fbuild._build_marshal(False, False)
    assert len(runs) == 2


def test_extension_module_is_built_again_for_newer_sources(runs, monkeypatch, tmp_path):
    source = tmp_path / "marshal.cpp"
    source.write_text("")
    monkeypatch.setattr(fbuild, "MARSHAL_SRC", str(source))
    fbuild._build_marshal(False, False)
    later = os.path.getmtime(fbuild.MARSHAL) + 10
    os.utime(source, (later, later))
    fbuild._build_marshal(False, False)
    assert len(runs) == 2
