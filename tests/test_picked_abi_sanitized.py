"""The refusals of the router, experts and adapters again, against the build whose
host code carries AddressSanitizer and UndefinedBehaviorSanitizer (no GPU)."""
import os
import subprocess
import sys

from mxfp4_block_scaled_02_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_refusals_under_asan_and_ubsan():
    lib = build.build_sanitized(verbose=False)
    env = dict(os.environ, LD_PRELOAD=build.sanitizer_runtime(), MXFP4_LIB=lib,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_picked_abi.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert " passed" in out
