"""The host code of the 8-bit product and the cross entropy (argument checks,
routing, planning) under the address and undefined-behaviour sanitizers: built
by the host compiler with stand-in launchers, and their CPU tests run against
that build."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matmul_pack_b1_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.slow
def test_f8_and_xent_tests_under_asan_and_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("needs g++ and the HIP headers")
    asan = subprocess.run([gxx, "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    if not (os.path.isabs(asan) and os.path.exists(asan)):
        pytest.skip("no libasan for this compiler")
    lib = str(tmp_path / "libhyb_sanitized.so")
    sources = [os.path.join(CSRC, f) for f in ("hyb_api.cpp", "hyb_route.cpp", "hyb_f8_api.cpp", "hyb_f8_route.cpp",
                                               "hyb_xent_api.cpp", "hyb_xent_plan.cpp")]
    sources += [os.path.join(ROOT, "tests", f) for f in ("sanitize_launch_stub.cpp", "sanitize_f8_stub.cpp")]
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
           "-o", lib, *sources, f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    env = dict(os.environ)
    env.update({
        "HYB_LIB": lib,
        "LD_PRELOAD": asan,
        "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1",
        "UBSAN_OPTIONS": "print_stacktrace=1:halt_on_error=1",
    })
    run = subprocess.run([sys.executable, "-m", "pytest", os.path.join(ROOT, "tests", "test_f8_cpu.py"),
                          os.path.join(ROOT, "tests", "test_xent_cpu.py"), "-q", "-x", "-p", "no:cacheprovider",
                          "-m", "not gpu"], capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    tail = (run.stdout + run.stderr)[-4000:]
    assert run.returncode == 0, tail
    assert "passed" in run.stdout and "ERROR: AddressSanitizer" not in tail and "runtime error" not in tail, tail
