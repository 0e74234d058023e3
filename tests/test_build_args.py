"""The build's optional part, _latent_args.so, with compilers that only say what they were asked."""
import os
import subprocess
import types

import pytest

from kda_gated_delta_04_gb300 import build


@pytest.fixture
def bench(monkeypatch, tmp_path):
    """The build module over an empty folder.  `ran`: the commands; `fails(cmd)`: which of them fail."""
    state = types.SimpleNamespace(ran=[], fails=lambda cmd: False, lib=str(tmp_path / "libkda.so"),
                                  args=str(tmp_path / "_latent_args.so"), build=build.build)

    def run(cmd, **kw):
        state.ran.append(cmd)
        if state.fails(cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "no such luck")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(" ".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "LIB_PATH", state.lib)
    monkeypatch.setattr(build, "ARGS_PATH", state.args)
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(build.subprocess, "run", run)
    return state


def compiling(cmd):
    return cmd[0] == "g++" and "-c" in cmd


def linking(cmd):
    return cmd[0] == "g++" and "-shared" in cmd


def absent(cmd):
    if cmd[0] == "g++":
        raise FileNotFoundError("g++")
    return False


def test_both_are_built(bench):
    bench.build()
    assert os.path.exists(bench.lib) and os.path.exists(bench.args)


@pytest.mark.parametrize("fails", [compiling, linking, absent])
def test_the_optional_part_does_not_fail_the_build(bench, capfd, fails):
    """Where g++ is missing or cannot compile or link it (a torch without CUDA's libraries), the library is
    built all the same, and the reason is said."""
    bench.fails = fails
    assert bench.build() == bench.lib and os.path.exists(bench.lib) and not os.path.exists(bench.args)
    assert "_latent_args left out" in capfd.readouterr().err


@pytest.mark.parametrize("missing", ["Python.h", "python_variable.h", "CUDAStream.h", "libc10_cuda.so"])
def test_what_it_needs_is_asked_for_first(bench, capfd, monkeypatch, missing):
    there = os.path.exists
    monkeypatch.setattr(build.os.path, "exists", lambda p: not p.endswith(missing) and there(p))
    assert bench.build() == bench.lib
    assert not any(cmd[0] == "g++" for cmd in bench.ran) and not there(bench.args)
    assert missing in capfd.readouterr().err


@pytest.mark.parametrize("fails", [compiling, linking, absent])
def test_an_old_module_does_not_stay_beside_a_new_library(bench, fails):
    """Its calls could have other arguments."""
    bench.build()
    assert os.path.exists(bench.args)
    bench.fails = fails
    try:
        bench.build(force=True)
    except (RuntimeError, FileNotFoundError):
        pass
    assert not os.path.exists(bench.args)


def test_no_old_module_while_the_library_is_replaced(bench, monkeypatch):
    bench.build()
    seen = []
    replace = os.replace
    monkeypatch.setattr(build.os, "replace", lambda a, b: (seen.append(b == bench.lib and os.path.exists(bench.args)), replace(a, b)))
    bench.build(force=True)
    assert seen and not any(seen)


def test_nothing_runs_when_all_is_there(bench):
    bench.build()
    bench.ran.clear()
    bench.build()
    assert not bench.ran


def test_a_missing_module_is_built_again(bench):
    """By itself: the library stays as it is."""
    bench.build()
    os.remove(bench.args)
    bench.ran.clear()
    bench.build()
    assert os.path.exists(bench.args) and [cmd[0] for cmd in bench.ran] == ["g++", "g++"]


def test_a_module_for_another_torch_is_built_again(bench, monkeypatch):
    bench.build()
    before = os.path.getmtime(bench.lib)
    monkeypatch.setattr(build, "_torch_version", lambda: "1.0", raising=False)
    bench.ran.clear()
    bench.build()
    assert [cmd[0] for cmd in bench.ran] == ["g++", "g++"] and os.path.getmtime(bench.lib) == before
    bench.ran.clear()
    bench.build()
    assert not bench.ran


def test_a_module_left_out_is_not_tried_on_every_call(bench, capfd):
    """But the reason is said again, and another torch is another chance."""
    bench.fails = compiling
    bench.build()
    bench.ran.clear()
    capfd.readouterr()
    bench.build()
    assert not bench.ran and "_latent_args left out" in capfd.readouterr().err


def test_a_changed_module_source_leaves_the_library(bench, monkeypatch, tmp_path):
    bench.build()
    src = tmp_path / "changed.cpp"
    src.write_text("")
    os.utime(src, (os.path.getmtime(bench.lib) + 10,) * 2)
    monkeypatch.setattr(build, "ARGS_SRC", str(src))
    bench.ran.clear()
    bench.build()
    assert [cmd[0] for cmd in bench.ran] == ["g++", "g++"]


def test_a_module_to_build_without_nvcc(bench, monkeypatch, capfd):
    """The library is there; what the module's headers need is not."""
    bench.build()
    os.remove(bench.args)

    def none():
        raise RuntimeError("nvcc not found")

    monkeypatch.setattr(build, "nvcc_path", none)
    assert bench.build() == bench.lib and "nvcc not found" in capfd.readouterr().err
