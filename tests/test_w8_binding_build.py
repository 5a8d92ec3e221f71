"""When the binding's native part is built, and what a call does where it cannot be."""
import os

import pytest
import torch

from gemv_w4a16_groupwise_b200 import build


@pytest.fixture
def compiled(monkeypatch):
    """The commands that the build would run, each leaving the file that it is asked for; files made are removed."""
    build.build_binding()
    commands, made = [], []

    def run(cmd, check):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        commands.append(cmd)
        return None

    real = os.replace
    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build.os, "replace", lambda a, b: (made.append(b), real(a, b)))
    yield commands
    for path in made:
        os.unlink(path)


@pytest.mark.parametrize("what,value", [("__version__", "9.9.9"), ("_C._GLIBCXX_USE_CXX11_ABI", None)])
def test_another_torch_gets_its_own_binary(monkeypatch, compiled, what, value):
    build.build_binding()
    assert not compiled                        # up to date
    owner, name = (torch._C, what[3:]) if what.startswith("_C.") else (torch, what)
    monkeypatch.setattr(owner, name, not getattr(owner, name) if value is None else value)
    first = build.build_binding()
    assert len(compiled) == 1
    assert build.build_binding() == first and len(compiled) == 1


def test_changed_source_with_an_old_date_is_built(monkeypatch, compiled, tmp_path):
    source = tmp_path / "w8_native.cpp"
    source.write_bytes(open(build.BINDING, "rb").read() + b"\n// changed\n")
    os.utime(source, (1, 1))
    build.build_binding()
    assert not compiled
    monkeypatch.setattr(build, "BINDING", str(source))
    build.build_binding()
    assert len(compiled) == 1
