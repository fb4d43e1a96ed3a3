"""The build step's decisions, with the compilers replaced: what is stale, and what a missing torch or
a binding that does not compile leaves."""
from __future__ import annotations

import os
import subprocess
import warnings

import pytest

from blackwell_tensor_core_fp16_gb300 import _build


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    """Commands write their output; `fails` refuses those that name one of its words."""
    for name in ("LIB_PATH", "BINDING_PATH", "BINDING_ABI"):
        monkeypatch.setattr(_build, name, str(tmp_path / os.path.basename(getattr(_build, name))))
    monkeypatch.setattr(_build, "PKG_DIR", str(tmp_path))
    fails, calls = set(), []

    def run(cmd, **kw):
        calls.append(cmd)
        bad = any(word in " ".join(cmd) for word in fails)
        if not bad:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, int(bad), "", "no" if bad else "")

    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build.subprocess, "Popen", None)
    run.fails, run.calls, run.made = fails, calls, lambda: sorted(os.listdir(tmp_path))
    return run


BOTH = ["_decode.so", "_decode.so.abi", "libgemm_f16.so"]


def test_build_and_build_again(compilers):
    assert _build.is_stale()
    _build.build()
    assert compilers.made() == BOTH and not _build.is_stale()
    before = len(compilers.calls)
    _build.build()
    assert len(compilers.calls) == before
    _build.build(force=True)
    assert len(compilers.calls) == 2 * before and compilers.made() == BOTH


def test_without_torch_the_library_is_built(compilers, monkeypatch):
    monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name: None)
    monkeypatch.setitem(__import__("sys").modules, "torch", None)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        _build.build()
    assert compilers.made() == ["libgemm_f16.so"] and not _build.is_stale()


@pytest.mark.parametrize("change", ["torch", "python"])
def test_another_torch_or_python_makes_the_binding_stale(compilers, monkeypatch, change):
    _build.build()
    if change == "torch":
        monkeypatch.setattr(_build.importlib.metadata, "version", lambda name: "9.9")
    else:
        monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda name: "cpython-399")
    assert _build.is_stale()
    before = len(compilers.calls)
    _build.build()
    assert not _build.is_stale()
    assert [c[0] for c in compilers.calls[before:]] == ["g++", "g++"]     # the library stands


@pytest.mark.parametrize("word", ["decode_binding.cpp", "-ltorch_python"], ids=["compile", "link"])
def test_a_binding_that_does_not_compile_leaves_the_library(compilers, word):
    compilers.fails.add(word)
    with pytest.warns(RuntimeWarning, match="_decode.so is not built"):
        _build.build()
    assert compilers.made() == ["libgemm_f16.so"]
    assert _build.is_stale()                       # it is tried again
    compilers.fails.clear()
    _build.build()
    assert compilers.made() == BOTH


def test_no_compiler_for_the_binding(compilers, monkeypatch):
    run = _build.subprocess.run

    def missing(cmd, **kw):
        if cmd[0] == "g++":
            raise FileNotFoundError(2, "No such file or directory", "g++")
        return run(cmd, **kw)

    monkeypatch.setattr(_build.subprocess, "run", missing)
    with pytest.warns(RuntimeWarning, match="g[+][+]"):
        _build.build()
    assert compilers.made() == ["libgemm_f16.so"]


@pytest.mark.parametrize("word", ["gdn_step.cu", "-shared"], ids=["compile", "link"])
def test_a_library_that_does_not_compile_leaves_nothing(compilers, word):
    compilers.fails.add(word)
    with pytest.raises(RuntimeError, match="failed"):
        _build.build()
    assert compilers.made() == []
