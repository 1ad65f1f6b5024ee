"""The paged cache's, paged attention's and the gated norm's host code and refusals under
AddressSanitizer and UndefinedBehaviorSanitizer, as tests/test_sanitized_block.py
does for the block operators'."""
import os
import shutil
import subprocess
import sys

import pytest

from rank_gemm_svdq_amd import build as BLD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++ with the sanitizer runtimes")
def test_serving_host_code_is_clean_under_asan_and_ubsan():
    lib = BLD.build(sanitize=True, reuse_device_objects=True)
    env = dict(os.environ, SVDQ_TEST_LIB=lib, **BLD.sanitizer_env())
    env.pop("PYTEST_XDIST_WORKER", None)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:xdist", "-m", "not gpu",
                        os.path.join(ROOT, "tests", "test_serving_refusals.py")],
                       cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=1200)
    assert r.returncode == 0 and " passed" in r.stdout and " failed" not in r.stdout, r.stdout[-3000:]
    assert "AddressSanitizer" not in r.stdout and "runtime error" not in r.stdout, r.stdout[-3000:]
