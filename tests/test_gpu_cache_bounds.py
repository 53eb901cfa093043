"""The paged cache's suites under the bounds-checking build: every access of its
kernels to the pool, the table, the lists, the workspaces, queries and outputs is
checked against its buffer, and each test's device status has to stay zero."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUITES = ["tests/test_gpu_cache.py", "tests/test_gpu_cache_edges.py", "tests/test_gpu_window_edges.py"]


def test_cache_suites_under_the_bounds_checking_build(lib):
    from io_aware_exact_20_b200 import build
    env = dict(os.environ, FA_B200_LIBRARY=build.build_variant("bounds"))
    env["PYTHONPATH"] = os.pathsep.join([os.path.join(ROOT, "tests"), env.get("PYTHONPATH", "")])
    probe = "import io_aware_exact_20_b200 as fa; assert fa.library().fa_debug_bounds_checking() == 1"
    subprocess.run([sys.executable, "-c", probe], cwd=ROOT, env=env, check=True, timeout=300)
    r = subprocess.run([sys.executable, "-m", "pytest", *SUITES, "-m", "gpu", "-q", "-x", "-p", "device_status",
                        "-p", "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
