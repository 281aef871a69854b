"""The build's order on the host: the C library needs hipcc alone, and is there
whatever becomes of the Python binding. The compilers are replaced by stubs."""
import os

import pytest

from matrix_aware_optimizers_amd import build as b


@pytest.fixture
def stubs(monkeypatch, tmp_path):
    monkeypatch.setattr(b, "OBJ", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmao.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_layers.so"))
    monkeypatch.setattr(b, "HIPCC", os.devnull)
    monkeypatch.setattr(b, "_compile", lambda src: src)
    (tmp_path / "_layers.so").write_text("of an older library")

    def run(cmd, what):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(what)

    monkeypatch.setattr(b, "_run", run)
    return tmp_path


def test_library_and_binding(stubs):
    pytest.importorskip("torch")
    assert b.build() == b.LIB
    assert (stubs / "libmao.so").read_text() == "link of libmao.so"
    assert (stubs / "_layers.so").read_text() == "link of _layers.so"


@pytest.mark.parametrize("lacks", ["g++", "headers"])
def test_library_alone(stubs, monkeypatch, capsys, lacks):
    if lacks == "g++":
        monkeypatch.setattr(b.shutil, "which", lambda name: None)
    else:
        monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(stubs / "nowhere")})
    if lacks == "headers":
        pytest.importorskip("torch")
    assert b.build() == b.LIB
    assert (stubs / "libmao.so").exists()
    assert not (stubs / "_layers.so").exists()  # an old one does not fit the new library
    assert lacks in capsys.readouterr().err.replace("Python's headers", "headers")


def test_library_is_there_when_the_binding_fails(stubs, monkeypatch):
    pytest.importorskip("torch")

    def broken():
        raise RuntimeError("g++ on binding.cpp failed")

    monkeypatch.setattr(b, "_compile_binding", broken)
    with pytest.raises(RuntimeError, match="binding"):
        b.build()
    assert (stubs / "libmao.so").exists() and not (stubs / "_layers.so").exists()
