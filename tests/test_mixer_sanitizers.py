"""The C ABI of the gated delta rule and of the group norm under AddressSanitizer
and UndefinedBehaviorSanitizer, on the CPU: its refusals run in a child process
that loads the library built with the host code instrumented."""
import os
import subprocess
import sys

import pytest

from selective_scan_ssm_amd import build
from test_sanitizers import CLANG, ROOT, asan_runtime


def test_refusals_run_clean(tmp_path):
    rt = asan_runtime()
    if rt is None or not os.path.exists(CLANG):
        pytest.skip("no clang AddressSanitizer runtime in this image")
    lib = build.build_host_sanitized(str(tmp_path / "libssmscan_asan.so"))
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1", SSM_SCAN_LIB=lib, PYTHONDONTWRITEBYTECODE="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "tests/test_mixer_abi.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert "ERROR: AddressSanitizer" not in tail and "runtime error" not in tail, tail
