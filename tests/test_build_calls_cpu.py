"""The C++ part of the binding and the torch it is compiled for: another torch
or another command means another build, and a build for another torch is not
imported."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import textwrap

import pytest
import torch

from paged_kv_cache_316_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def started(monkeypatch, tmp_path):
    """Commands that the build would start; what it makes lies in tmp_path."""
    commands = []

    class Started:
        returncode = 0

        def __init__(self, cmd, **kw):
            commands.append(cmd)
            open(cmd[cmd.index("-o") + 1], "w").close()

        def communicate(self):
            return "", None

    monkeypatch.setattr(build, "LIB_CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "CALLS_STAMP", str(tmp_path / "calls.stamp"))
    monkeypatch.setattr(build.subprocess, "Popen", Started)

    def run():
        n = len(commands)
        build._finish_calls(build._start_calls(False))
        return commands[n:]
    return run


def test_another_torch_is_another_build(started, monkeypatch):
    first = started()
    assert len(first) == 1 and any(torch.__version__ in x for x in first[0])
    assert started() == [] and started() == []
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    again = started()
    assert len(again) == 1 and any("9.9.9" in x for x in again[0])
    assert started() == []


def test_other_paths_are_another_build(started, monkeypatch):
    assert len(started()) == 1
    monkeypatch.setattr(torch, "__file__", "/elsewhere/torch/__init__.py")
    assert len(started()) == 1 and started() == []


def test_no_stamp_is_another_build(started):
    assert len(started()) == 1
    os.remove(build.CALLS_STAMP)
    assert len(started()) == 1 and started() == []


def test_the_name_carries_the_interpreter():
    assert os.path.basename(build.LIB_CALLS) == "_calls" + sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.exists(build.LIB_CALLS)


def test_a_build_for_another_torch_is_refused():
    run = subprocess.run([sys.executable, "-c", textwrap.dedent("""
        import torch
        import paged_kv_cache_316_gb300 as pk
        real, torch.__version__ = torch.__version__, "9.9.9"
        try:
            pk.paged_merge_states([])
        except pk.PagedKVError as e:
            assert "built for torch " + str(real) in str(e) and "9.9.9" in str(e), e
        else:
            raise AssertionError("went through")
        assert pk.paged_decode_workspace_size(4, 1, 8, 2, 128, 100, 16) >= 0  # the library alone
        torch.__version__ = real
        try:
            pk.paged_merge_states([])
        except pk.PagedKVError as e:
            assert "no states" in str(e), e
    """)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr
