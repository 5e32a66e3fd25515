"""The C library is built on a host without torch; only the binding of the
layer operators to torch is left out."""

import importlib.util

from blockwise_bit_codebook_amd import build


def test_no_binding_without_torch(monkeypatch, capsys):
    commands = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    monkeypatch.setattr(build, "_compile", lambda src, verbose: src)
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: commands.append(cmd) or Done())
    monkeypatch.setattr(build.shutil, "move", lambda a, b: None)
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build() == build.LIB
    assert [c[0] for c in commands] == [build.HIPCC] and "not built" in capsys.readouterr().out
    monkeypatch.undo()
    if importlib.util.find_spec("torch") is not None:
        commands.clear()
        monkeypatch.setattr(build, "_compile", lambda src, verbose: src)
        monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: commands.append(cmd) or Done())
        monkeypatch.setattr(build.shutil, "move", lambda a, b: None)
        build.build()
        assert [c[0] for c in commands] == [build.HIPCC, "g++"]
