"""The host side of the training-gradient entry points under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU): validation, planning and workspace layout of
``grads.cpp``, by the tests that need no GPU.  Any sanitizer report fails the test."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_training_host_suites_under_asan_and_ubsan(tmp_path):
    from matrix_optimizer_muon_amd import build_sanitized as bs
    lib = bs.build(str(tmp_path))
    env = dict(os.environ, LD_PRELOAD=bs.asan_runtime(), DMUON_LIBRARY=lib,
               ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                        os.path.join("tests", "test_training_host.py"),
                        os.path.join("tests", "test_training_sizes_host.py")], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=900)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert " passed" in r.stdout
