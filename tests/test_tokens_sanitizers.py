"""The host code of sampling, the embedding and the orthogonalised update under AddressSanitizer and UndefinedBehaviorSanitizer, with the library that
tests/test_host_sanitizers.py builds (device code as usual, CPU only)."""
import glob
import os
import subprocess
import sys

import pytest

from second_order_optimizer_amd import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not installed")
def test_tokens_abi_under_asan_and_ubsan():
    S = pytest.importorskip("tests.test_host_sanitizers")
    rt = S._asan_runtime()
    if not os.path.isabs(rt) or not os.path.exists(rt):
        pytest.skip("clang AddressSanitizer runtime not found")
    srcs = glob.glob(os.path.join(B.CSRC, "*")) + glob.glob(os.path.join(ROOT, "include", "*"))
    fresh = os.path.exists(S.SAN_LIB) and all(os.path.getmtime(s) < os.path.getmtime(S.SAN_LIB) for s in srcs)
    lib = S.SAN_LIB if fresh else S._build()
    env = dict(os.environ, KFAC_LIBRARY=lib, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                        os.path.join(ROOT, "tests", "test_tokens_abi.py")],
                       cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:]
    assert "AddressSanitizer" not in r.stdout and "runtime error:" not in r.stdout, r.stdout[-4000:]
    assert " passed" in r.stdout and " failed" not in r.stdout, r.stdout[-2000:]
