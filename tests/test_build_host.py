"""The build's steps with stand-ins for the compilers (no CUDA, no GPU): what is built when torch or its compiler is
missing, and what makes the binding out of date."""
import importlib.metadata
import os
import stat
import sys
import sysconfig

import pytest

FAKE_CC = """#!/bin/sh
# writes the file named behind -o and counts the call
echo "$0" >> "{log}"
[ -e "{log}.fail.$(basename "$0")" ] && exit 1
while [ $# -gt 0 ]; do
  if [ "$1" = -o ]; then echo built > "$2"; fi
  shift
done
"""


@pytest.fixture()
def b(tmp_path, monkeypatch):
    """The build module with its outputs, sources and compilers below tmp_path; b.runs() lists the compilers' calls."""
    from microscaling_fp4_quantized_b200 import build
    csrc, include = tmp_path / "csrc", tmp_path / "include"
    csrc.mkdir()
    include.mkdir()
    (csrc / "one.cu").write_text("")
    (csrc / "binding.cpp").write_text("")
    (include / "sage_fp4.h").write_text("")
    log = tmp_path / "log"
    for name in ("nvcc", "cxx"):
        cc = tmp_path / name
        cc.write_text(FAKE_CC.format(log=log))
        cc.chmod(cc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("NVCC", str(tmp_path / "nvcc"))
    monkeypatch.setenv("CXX", str(tmp_path / "cxx"))
    for name, value in (("PKG", tmp_path), ("CSRC", csrc), ("INCLUDE", include), ("BUILD", tmp_path / "_build"),
                        ("LIB", tmp_path / "lib.so"), ("LIB_CHECKS", tmp_path / "lib_checks.so"),
                        ("BINDING", tmp_path / "_binding.so")):
        monkeypatch.setattr(build, name, str(value))

    def runs():
        calls = log.read_text().split() if log.exists() else []
        log.write_text("")
        return [os.path.basename(c) for c in calls]

    def fail(name):
        (tmp_path / f"log.fail.{name}").write_text("")

    monkeypatch.setattr(build, "runs", runs, raising=False)
    monkeypatch.setattr(build, "fail", fail, raising=False)
    return build


def test_everything_is_built_once(b):
    assert b.build() == b.LIB and os.path.exists(b.LIB) and os.path.exists(b.BINDING)
    assert sorted(b.runs()) == ["cxx", "nvcc", "nvcc"]
    b.build()
    assert b.runs() == []
    b.build(force=True)
    assert sorted(b.runs()) == ["cxx", "nvcc", "nvcc"]


def test_the_library_is_built_without_torch(b, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.BINDING) and "torch" in capsys.readouterr().err
    assert set(b.runs()) == {"nvcc"}


def test_the_library_is_there_when_the_binding_does_not_build(b):
    b.fail("cxx")
    with pytest.raises(RuntimeError, match="binding"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)


@pytest.mark.parametrize("change", ["torch", "python", "source"])
def test_the_binding_follows_what_it_was_built_for(b, monkeypatch, tmp_path, change):
    """Its file is newer than its sources and yet of no use to another torch or Python (their C++ and C interfaces)."""
    b.build()
    b.runs()
    if change == "torch":
        monkeypatch.setattr(importlib.metadata, "version", lambda name: "99.0")
    elif change == "python":
        monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-x86_64-linux-gnu")
    else:
        later = os.path.getmtime(b.BINDING) + 10
        os.utime(tmp_path / "csrc" / "binding.cpp", (later, later))
    b.build()
    assert [r for r in b.runs() if r.startswith("cxx")] == ["cxx"]
    if change != "source":  # (its time stays ahead of the stand-in's output)
        b.build()
        assert [r for r in b.runs() if r.startswith("cxx")] == []
