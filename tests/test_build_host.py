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
    for name, file in (("BUILD", ""), ("LIB", "libpe.so"), ("BIND", "pe_bind.so"), ("BIND_FOR", "pe_bind.for")):
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


def _torch_of(monkeypatch, folder, version):
    """A torch of this version in this folder, as far as the build looks at it."""
    os.makedirs(folder, exist_ok=True)
    with open(os.path.join(folder, "version.py"), "w") as f:
        f.write(f"__version__ = {version!r}\n")
    monkeypatch.setattr(B, "_torch", lambda: folder)


def test_another_torch_or_python_compiles_the_binding_again(built, tmp_path, monkeypatch):
    one, two = str(tmp_path / "one"), str(tmp_path / "two")
    _torch_of(monkeypatch, one, "2.9.1")
    assert sorted(built()) == ALL and built() == [] and B.bind_is_current()
    _torch_of(monkeypatch, one, "2.11.0")                       # upgraded in its place
    assert not B.bind_is_current() and built() == ["pe_bind.so"] and built() == []
    _torch_of(monkeypatch, two, "2.11.0")                       # the same version elsewhere, built otherwise perhaps
    assert built() == ["pe_bind.so"] and built() == []
    abi = B.sysconfig.get_config_var
    monkeypatch.setattr(B.sysconfig, "get_config_var", lambda name: "cpython-399" if name == "SOABI" else abi(name))
    assert built() == ["pe_bind.so"] and built() == [] and B.bind_is_current()
    os.remove(B.BIND_FOR)                                       # a build that ended early, or an older one
    assert built() == ["pe_bind.so"] and B.bind_is_current()
    os.remove(B.BIND)
    assert not B.bind_is_current() and built() == ["pe_bind.so"]


def test_the_built_binding_is_for_this_torch():
    import torch

    import speculative_decoding_step_gb300 as pe

    pe._binding()
    with open(B.BIND_FOR) as f:
        stamp = f.read()
    assert B.bind_is_current() and os.path.dirname(torch.__file__) in stamp and torch.__version__.split("+")[0] in stamp
