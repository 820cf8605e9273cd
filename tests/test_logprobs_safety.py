"""The host side of the log-probability and clipping entry points (CPU): their suites under
AddressSanitizer and UndefinedBehaviorSanitizer, and every call with each of its allocations
failing (see tests/c/no_throw_logprobs.cpp)."""
import os
import subprocess
import sys

from matrix_optimizer_muon_amd import _binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_host_suites_under_asan_and_ubsan(tmp_path):
    from matrix_optimizer_muon_amd import build_sanitized as bs
    lib = bs.build(str(tmp_path))
    env = dict(os.environ, LD_PRELOAD=bs.asan_runtime(), DMUON_LIBRARY=lib,
               ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                        os.path.join("tests", "test_logprobs_host.py"), os.path.join("tests", "test_clip_host.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert " passed" in r.stdout


def test_failing_allocations_become_error_codes(tmp_path):
    B.lib()
    exe = str(tmp_path / "no_throw")
    here = os.path.dirname(B.LIB_PATH)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-rdynamic", "-I", os.path.join(ROOT, "include"),
                        os.path.join(ROOT, "tests", "c", "no_throw_logprobs.cpp"), "-o", exe, B.LIB_PATH, f"-Wl,-rpath,{here}",
                        "-Wl,-rpath,/opt/rocm/lib", "-Wl,-rpath-link,/opt/rocm/lib"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], env=dict(os.environ, DMUON_TEST_FAIL_AT="plan"), capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), (r.returncode, r.stdout, r.stderr)
    counts = [int(line.split(": ")[1].split()[0]) for line in r.stdout.splitlines()[:-1]]
    assert len(counts) == 16 and sum(n > 0 for n in counts) >= 10, r.stdout
