"""What loads when: append, decode and prefill need the C library alone; the
C++ part of the binding (_calls.so, bound to one interpreter and one torch) is
asked for by the calls that go through it, and a failure to load it stays an
error that says so."""
from __future__ import annotations

import os
import subprocess
import sys
import textwrap

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    run = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr
    return run.stdout


def test_without_the_cpp_part():
    python("""
        import sys, torch
        import paged_kv_cache_316_gb300 as pk
        sys.modules["paged_kv_cache_316_gb300._calls"] = None  # as if it could not be imported
        assert pk.paged_decode_workspace_size(4, 1, 8, 2, 128, 100, 16) >= 0 and not pk.debug_bounds()
        assert pk.paged_decode_shared_workspace_size(4, 1, 8, 2, 128, 1, 100, 100, 16) > 0
        x = torch.zeros(1, 8, 64, dtype=torch.half)
        for _ in range(2):  # every time
            for call in (lambda: pk.paged_merge_states([(x, x[..., 0].float())]),
                         lambda: pk.paged_rotary(x, x, torch.zeros(1, dtype=torch.int32), torch.ones(32).double())):
                try:
                    call()
                except pk.PagedKVError as e:
                    assert "_calls.so" in str(e)
                else:
                    raise AssertionError("went through")
        assert pk.paged_decode_workspace_size(4, 1, 8, 2, 128, 100, 16) >= 0
    """)


def test_a_first_hand_over_that_fails():
    python("""
        import sys, types, torch
        import paged_kv_cache_316_gb300 as pk
        from paged_kv_cache_316_gb300 import binding
        broken = types.ModuleType("paged_kv_cache_316_gb300._calls")
        def use(*a):
            raise RuntimeError("not today")
        broken.use = use
        sys.modules["paged_kv_cache_316_gb300._calls"] = broken
        pk._calls = broken
        for _ in range(2):
            try:
                pk.paged_merge_states([])
            except RuntimeError as e:
                assert "not today" in str(e)
            else:
                raise AssertionError("went through")
            assert binding._calls is None
        del sys.modules["paged_kv_cache_316_gb300._calls"], pk._calls
        try:
            pk.paged_merge_states([])
        except pk.PagedKVError as e:
            assert "no states" in str(e)
    """)


def test_many_threads_at_first():
    python("""
        import threading, torch
        import paged_kv_cache_316_gb300 as pk
        got, go = [], threading.Barrier(16)
        def first():
            go.wait()
            try:
                pk.paged_merge_states([])
            except BaseException as e:
                got.append(repr(e))
        threads = [threading.Thread(target=first) for _ in range(16)]
        [t.start() for t in threads]
        [t.join() for t in threads]
        assert len(got) == 16 and all("PagedKVError" in g and "no states" in g for g in got), got
    """)


def test_switching_builds():
    python("""
        import paged_kv_cache_316_gb300 as pk
        from paged_kv_cache_316_gb300 import binding
        try:
            pk.paged_merge_states([])
        except pk.PagedKVError:
            pass
        handed = []
        real = binding._calls
        class Spy:
            def use(self, *a):
                handed.append(a)
                real.use(*a)
        binding._calls = Spy()
        binding.load_library(binding.library_path())  # every build that is loaded is handed over
        assert len(handed) == 1 and all(handed[0][2:])
    """)
