"""No C++ exception leaves the training-gradient entry points when the host runs out of
memory: each call with each of its allocations failing (CPU; see tests/c/no_throw.cpp)."""
import os
import subprocess

from matrix_optimizer_muon_amd import _binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_failing_allocations_become_error_codes(tmp_path):
    B.lib()
    exe = str(tmp_path / "no_throw")
    here = os.path.dirname(B.LIB_PATH)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-rdynamic", "-I", os.path.join(ROOT, "include"),
                        os.path.join(ROOT, "tests", "c", "no_throw.cpp"), "-o", exe, B.LIB_PATH, f"-Wl,-rpath,{here}",
                        "-Wl,-rpath,/opt/rocm/lib", "-Wl,-rpath-link,/opt/rocm/lib"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], env=dict(os.environ, DMUON_TEST_FAIL_AT="plan"), capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), (r.returncode, r.stdout, r.stderr)
    # the calls that plan and those that refuse do allocate
    counts = [int(l.split(": ")[1].split()[0]) for l in r.stdout.splitlines()[:-1]]
    assert len(counts) == 16 and sum(n > 0 for n in counts) >= 10, r.stdout
