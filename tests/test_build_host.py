"""What the build compiles, and when (no GPU, and no compiler: commands are recorded and their outputs made up)."""

import importlib
import importlib.util
import os
import subprocess

import pytest

B = importlib.import_module("speculative_decoding_step_gb300.build")


@pytest.fixture
def built(tmp_path, monkeypatch):
    """build() in a folder of its own: returns the commands of a call."""
    for name, file in (("BUILD", ""), ("LIB", "libpe.so"), ("BIND", "pe_bind.so")):
        monkeypatch.setattr(B, name, os.path.join(str(tmp_path), file) if file else str(tmp_path))
    commands = []

    def run(cmd, **_):
        commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made up")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)

    def call(**kw):
        commands.clear()
        B.build(**kw)
        return [os.path.basename(c[c.index("-o") + 1]).split(".tmp")[0] for c in commands]

    return call


ALL = sorted([s.replace(".cu", ".o") for s in B.SOURCES] + ["libpe.so", "pe_bind.so"])


def test_everything_is_built_once(built):
    assert sorted(built()) == ALL
    assert built() == []
    assert sorted(built(force=True)) == ALL


def test_without_torch_the_library_is_built_alone(built, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert sorted(built()) == [n for n in ALL if n != "pe_bind.so"]
    assert built() == [] and os.path.exists(B.LIB) and not os.path.exists(B.BIND)
