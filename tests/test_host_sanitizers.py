"""The library's host code under AddressSanitizer and UndefinedBehavior-
Sanitizer, on the CPU: argument validation (abi.cpp) and the GEMM launch
planner (plan_gemm, plan_columns in gemm.hip).

1. The whole C-ABI argument matrix of tests/test_abi.py runs in a child
   Python process against a host-sanitized build of libfp8fg.so, with the
   sanitizer runtime preloaded; any sanitizer report fails the child.
2. A native driver sweeps the planner over shapes, expert counts, flags and
   CU counts under the same sanitizers and checks its invariants (column
   tiles cover N exactly, grids match the tile counts, each kernel only in
   its own case).
No GPU is involved: the planner makes no HIP call and every ABI call in the
matrix is rejected, or is a no-op, before any launch."""

import os
import subprocess
import sys

import pytest

from fp8_fine_grained_x1_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SAN_ENV = {
    "ASAN_OPTIONS": "detect_leaks=0:abort_on_error=0:halt_on_error=1",
    "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1",
}


@pytest.fixture(scope="module")
def sanitized():
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    lib, objs = build.build_host_sanitized()
    return lib, objs, build.asan_runtime()


def _env(runtime):
    env = dict(os.environ)
    env.update(SAN_ENV)
    env["LD_PRELOAD"] = runtime
    return env


def _no_reports(text):
    assert "ERROR: AddressSanitizer" not in text, text[-4000:]
    assert "runtime error:" not in text, text[-4000:]


def test_sanitized_library_is_instrumented(sanitized):
    lib, _, _ = sanitized
    out = subprocess.run(["nm", "-D", lib], capture_output=True, text=True).stdout
    assert "__asan_report_load8" in out and "__ubsan_handle" in out


def test_abi_matrix_under_sanitizers(sanitized):
    lib, _, runtime = sanitized
    code = ("import sys; sys.path.insert(0, %r); "
            "from fp8_fine_grained_x1_amd import binding as B; B.LIB_PATH = %r; "
            "import pytest; sys.exit(pytest.main(['-q', '-p', 'no:cacheprovider', %r]))"
            % (ROOT, lib, os.path.join(ROOT, "tests", "test_abi.py")))
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=_env(runtime),
                       capture_output=True, text=True, timeout=600)
    text = r.stdout + r.stderr
    _no_reports(text)
    assert r.returncode == 0, text[-4000:]
    assert " passed" in text and "failed" not in text


def test_planner_sweep_under_sanitizers(sanitized, tmp_path):
    _, objs, runtime = sanitized
    gemm_obj = [o for o in objs if os.path.basename(o) == "gemm.o"][0]
    src = os.path.join(ROOT, "tests", "native", "plan_check.cpp")
    obj = str(tmp_path / "plan_check.o")
    exe = str(tmp_path / "plan_check")
    cmd = ([build.HIPCC] + build.COMMON + build.DEVICE + build.HOST_SANITIZE +
           ["-x", "hip", "-c", src, "-o", obj])
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    rtdir = os.path.dirname(runtime)
    rtlib = os.path.basename(runtime)[len("lib"):-len(".so")]
    cmd = [build.HIPCC, "--offload-arch=gfx950", "-o", exe, obj, gemm_obj, "-L" + rtdir,
           "-l" + rtlib, "-Wl,-rpath," + rtdir]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], env=_env(runtime), capture_output=True, text=True, timeout=600)
    text = r.stdout + r.stderr
    _no_reports(text)
    assert r.returncode == 0, text[-4000:]
    assert " 0 failures" in text, text[-2000:]


def test_size_rules_under_sanitizers(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    runtime = build.asan_runtime()
    src = os.path.join(ROOT, "tests", "native", "size_check.cpp")
    obj, exe = str(tmp_path / "size_check.o"), str(tmp_path / "size_check")
    cmd = ([build.HIPCC] + build.COMMON + build.DEVICE + build.HOST_SANITIZE + ["-x", "hip", "-c", src, "-o", obj])
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    rtdir, rtlib = os.path.dirname(runtime), os.path.basename(runtime)[len("lib"):-len(".so")]
    cmd = [build.HIPCC, "--offload-arch=gfx950", "-o", exe, obj, "-L" + rtdir, "-l" + rtlib, "-Wl,-rpath," + rtdir]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], env=_env(runtime), capture_output=True, text=True, timeout=600)
    text = r.stdout + r.stderr
    _no_reports(text)
    assert r.returncode == 0 and "0 failures" in text, text[-4000:]
