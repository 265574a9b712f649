"""The build's order and what makes it stale, with the compilers replaced by stubs."""
import importlib.metadata
import os
import subprocess

import pytest

from selective_state_space_30_b200 import build


@pytest.fixture
def stubs(monkeypatch, tmp_path):
    """A build of two sources into tmp_path; the list of its steps."""
    steps = []
    csrc, include = tmp_path / "csrc", tmp_path / "include"
    csrc.mkdir(), include.mkdir()
    for f in ("a.cu", "b.cu", "front.cpp"):
        (csrc / f).write_text("")
    (include / "ssm_scan.h").write_text("")
    for k, v in dict(CSRC=csrc, INCLUDE=include, LIB=tmp_path / "lib.so", FRONT=tmp_path / "_front.so",
                     FRONT_STAMP=tmp_path / "_build" / "_front.txt", BUILD_DIR=tmp_path / "_build").items():
        monkeypatch.setattr(build, k, str(v))

    def compile_one(src, extra, build_dir=None):
        steps.append(os.path.basename(src))
        return src

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        steps.append("front" if os.path.basename(out).startswith("_front") else "link")
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "_compile", compile_one)
    monkeypatch.setattr(build.subprocess, "run", run)
    return steps


def _torch(monkeypatch, version):
    def found(name):
        if version is None:
            raise importlib.metadata.PackageNotFoundError(name)
        return version
    monkeypatch.setattr(build.importlib.metadata, "version", found)


def test_library_is_built_without_torch(monkeypatch, stubs):
    _torch(monkeypatch, None)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert sorted(stubs) == ["a.cu", "b.cu", "link"] and not os.path.exists(build.FRONT)


def test_library_is_linked_before_the_front_ends_fail(monkeypatch, stubs):
    _torch(monkeypatch, "9.9")

    def fail():
        raise RuntimeError("no headers")
    monkeypatch.setattr(build, "_compile_front", fail)
    with pytest.raises(RuntimeError, match="no headers"):
        build.build()
    assert os.path.exists(build.LIB) and "link" in stubs


def test_front_ends_follow_torch(monkeypatch, stubs):
    pytest.importorskip("torch")
    _torch(monkeypatch, "9.9")
    build.build()
    assert stubs[-2:] == ["link", "front"]
    del stubs[:]
    build.build()
    assert stubs == []                                   # nothing is stale
    _torch(monkeypatch, "9.10")
    build.build()
    assert stubs == ["front"]
    _torch(monkeypatch, None)
    build.build()
    assert stubs == ["front"]
