"""The shapes that the GPU tests run (route_shapes.py) reach every kernel, tile
and way of cutting of the 4-bit product and the gated projection: the library's
own route and plan are asked, through a few lines of C++ beside its headers."""
import ctypes
import itertools
import os
import shutil
import subprocess

import numpy as np
import pytest

import route_shapes as rs
from matmul_pack_b1_amd import binding as hb
from matmul_pack_b1_amd import gated

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
CUS = 256

ASK = r"""
#include "hyb_gated_internal.h"
#include "hyb_q4_internal.h"
extern "C" void ask_q4(int64_t n, int64_t k, int64_t m, int matrices, int64_t cus, int64_t* out) {
  const hyb::Q4Route r = hyb::q4_route(n, k, m, matrices, cus);
  out[0] = r.ap, out[1] = r.bp, out[2] = r.whole, out[3] = r.parts;
}
extern "C" void ask_gated(const hyb_gated_pair* w, int64_t m, int what, int64_t cus, int64_t* out) {
  const hyb::GatedPlan p = hyb::gated_plan(*w, m, what, cus);
  out[0] = p.bp, out[1] = p.whole, out[2] = p.parts, out[3] = p.small_dw, out[4] = p.both, out[5] = p.decode || p.rows;
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")):
        pytest.skip("needs g++ and the HIP headers")
    tmp = tmp_path_factory.mktemp("ask")
    src, so = str(tmp / "ask.cpp"), str(tmp / "libask.so")
    with open(src, "w") as f:
        f.write(ASK)
    csrc = os.path.join(ROOT, "matmul_pack_b1_amd", "csrc")
    res = subprocess.run([gxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
                          f"-I{csrc}", "-o", so, src, hb.LIB_PATH, f"-Wl,-rpath,{os.path.dirname(hb.LIB_PATH)}"],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    gated.lib()
    lib = ctypes.CDLL(so)
    I64, out = ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)
    lib.ask_q4.argtypes = [I64, I64, I64, ctypes.c_int, I64, out]
    lib.ask_gated.argtypes = [ctypes.POINTER(gated.HybGatedPair), I64, ctypes.c_int, I64, out]
    return lib


def q4_class(lib, matrices, n, k, m):
    out = (ctypes.c_int64 * 4)()
    lib.ask_q4(n, k, m, matrices, CUS, out)
    return matrices, out[0], out[1], out[2] > 0, out[3] > 1


def gated_plan(lib, n, k, m, what):
    layout, _ = hb.plan(n, k, 64, 64, "bf16", "idx2", np.arange(n // 64 * (k // 64)) % 2)
    pair = gated.HybGatedPair(ctypes.pointer(layout), None, ctypes.pointer(layout), None, None, None, n, k)
    out = (ctypes.c_int64 * 6)()
    lib.ask_gated(ctypes.byref(pair), m, what, CUS, out)
    assert not out[5]
    return list(out)


def test_q4_shapes(ask):
    for want, (n, k, m) in rs.Q4.items():
        assert q4_class(ask, want[0], n, k, m) == want, (n, k, m)
    for n, k, m in rs.Q4_NARROW:
        assert q4_class(ask, 1, n, k, m)[1] == q4_class(ask, 2, n, k, m)[1] == 16


def test_q4_shapes_are_all(ask):
    """No size of a wide grid takes a way that the shapes leave out."""
    sizes = (5, 40, 130, 300, 700, 1030, 2100, 4100, 6000, 8200, 12000, 28672)
    tokens = (5, 9, 17, 33, 65, 100, 200, 333, 520, 901, 1601, 2100, 4096)
    for matrices, n, k, m in itertools.product((1, 2), sizes, sizes, tokens):
        assert q4_class(ask, matrices, n, k, m) in rs.Q4, (matrices, n, k, m)


def forward_class(lib, n, k, m):
    p = gated_plan(lib, n, k, m, 0)
    return p[0], p[1] > 0, p[2] > 1


def backward_class(lib, n, k, m):
    p = gated_plan(lib, n, k, m, 3)
    return p[0], bool(p[4]), bool(p[3]), p[2] > 1


def test_gated_shapes(ask):
    for want, shape in rs.GATED_FORWARD.items():
        assert forward_class(ask, *shape) == want, shape
    for want, shape in rs.GATED_BACKWARD.items():
        assert backward_class(ask, *shape) == want, shape


def test_gated_shapes_are_all(ask):
    sizes = (64, 192, 512, 1024, 2816, 4096, 6400, 8192, 14336)
    for n, k, m in itertools.product(sizes, sizes, (129, 200, 333, 520, 901, 1301, 2050, 4096)):
        if n * k > 1 << 26:
            continue
        assert forward_class(ask, n, k, m) in rs.GATED_FORWARD, (n, k, m)
        assert backward_class(ask, n, k, m) in rs.GATED_BACKWARD, (n, k, m)
