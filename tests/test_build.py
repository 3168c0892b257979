"""The build script: what is built in which order and when, with the compilers replaced."""
import os
import subprocess

import pytest

from gqa_attention_rope_b200 import build as B


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """Targets in an empty folder; each "compiler" call is recorded and writes its output file."""
    calls = []

    def compile_(cmd):
        calls.append(cmd[0])
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
    for name, file in (("LIB", "lib.so"), ("BINDING", "_binding.so"), ("BINDING_STAMP", "_binding.torch")):
        monkeypatch.setattr(B, name, str(tmp_path / file), raising=False)
    monkeypatch.setattr(B, "binding_command", lambda out: ["g++", "-o", out])
    monkeypatch.setattr(subprocess, "check_call", compile_)
    return calls


def test_nothing_is_built_twice(sandbox):
    B.build()
    assert sorted(sandbox) == ["g++", "nvcc"]
    B.build()
    assert len(sandbox) == 2


def test_the_library_is_there_when_the_binding_fails(sandbox, monkeypatch):
    """A C program needs the library only: neither g++ nor torch's headers stand before it."""
    good = subprocess.check_call

    def no_gxx(cmd):
        if cmd[0] == "g++":
            raise subprocess.CalledProcessError(1, cmd)
        good(cmd)
    monkeypatch.setattr(subprocess, "check_call", no_gxx)
    with pytest.raises(subprocess.CalledProcessError):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


def test_another_torch_makes_the_binding_stale(sandbox, monkeypatch):
    B.build()
    monkeypatch.setattr(B, "_torch_version", lambda: "0.0.0", raising=False)
    B.build()
    assert sandbox.count("g++") == 2 and sandbox.count("nvcc") == 1
    B.build()
    assert len(sandbox) == 3
