"""The cache's and the description's host tests under AddressSanitizer and
UndefinedBehaviorSanitizer."""

import os
import subprocess
import sys

import pytest

from test_host_sanitizers import _env, _runtime

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_host_tests_under_asan_and_ubsan(lib):
    if _runtime("libasan.so") is None or _runtime("libubsan.so") is None:
        pytest.skip("the gcc sanitizer runtimes are not installed")
    from io_aware_exact_20_b200 import build
    env = _env(build.build_variant("sanitize"))
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_cache_edges_host.py", "tests/test_description_host.py",
                        "-q", "-p", "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    report = r.stdout[-3000:] + r.stderr[-3000:]
    assert r.returncode == 0, report
    assert "AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr, report
