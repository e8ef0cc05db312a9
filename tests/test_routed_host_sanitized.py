"""The argument checks of the routed experts' operators rerun against the
library whose host code is built with AddressSanitizer and
UndefinedBehaviorSanitizer, in a child process that preloads the ASan runtime."""
import os
import subprocess
import sys

import pytest

import test_host_sanitized as san
from bitplane_quantized_expert_amd import build


def test_routed_entry_points_under_asan_and_ubsan():
    rt = build.asan_runtime()
    if rt is None:
        pytest.skip("no ASan runtime next to hipcc")
    lib = build.ASAN_LIB
    newest = max(os.path.getmtime(s) for s in san.SOURCES)
    if not os.path.exists(lib) or os.path.getmtime(lib) < newest:
        build.build_sanitized()
    env = dict(os.environ, LD_PRELOAD=rt, PM_LIB=lib,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "not gpu", "-k", "not throws",
                        "-p", "no:cacheprovider", "tests/test_routed_host.py"],
                       cwd=san.ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = r.stdout[-4000:] + r.stderr[-4000:]
    assert r.returncode == 0, out
    assert "AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr, out
    assert " passed" in r.stdout, out
