"""A call that fails in its host set-up has enqueued nothing. The library's objects are linked against a stand-in for
the CUDA runtime (tests/csrc/fake_runtime.cpp) that counts launches and fails the call it is told to; every case is a
process of its own, in which the one-time set-up has not run."""
import glob
import json
import os
import subprocess
import sys

import pytest

from bwd_tri_attn_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))

CHILD = """
import ctypes, json, sys
path, name, d, fails = sys.argv[1:]
B, T, S, H, Hk, d = 2, 300, 1000, 4, 2, int(d)
class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "S", "H", "Hk", "d")] + [("scale", ctypes.c_float)] + [
        (n, ctypes.c_int64 * 3) for n in ("q", "k", "v")]
kv = (S * Hk * d, Hk * d, d)
shape = Shape(B, T, S, H, Hk, d, 0.125, (T * H * d, H * d, d), kv, kv)
lib = ctypes.CDLL(path)
pointers = {"tri_cross_fwd": 8, "tri_cross_bwd": 12}[name]
call = getattr(lib, name)
call.argtypes = [Shape] + [ctypes.c_void_p] * pointers + [ctypes.c_size_t, ctypes.c_void_p]
seen = []
for f in (fails, ""):
    lib.fake_fail(f.encode())
    seen += [call(shape, *[0x10000] * pointers, 1 << 34, None), lib.fake_launches()]
print(json.dumps(seen))
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    _build.build()
    objects = [os.path.join(_build.OBJDIR, os.path.basename(s)[:-3] + ".o") for s in glob.glob(os.path.join(_build.CSRC, "*.cu"))]
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    out = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-I", include, "-o", out, *objects, os.path.join(HERE, "csrc", "fake_runtime.cpp")],
                   check=True, capture_output=True)
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name,launches", [("tri_cross_fwd", 2), ("tri_cross_bwd", 5)])
@pytest.mark.parametrize("fails", ["cudaFuncSetAttribute", "cuTensorMapEncodeTiled", "cudaGetSymbolAddress", "cudaGetDevice",
                                   "cudaDeviceGetAttribute", "cudaSetDevice"])
def test_cross_attention(lib, name, launches, d, fails):
    r = subprocess.run([sys.executable, "-c", CHILD, lib, name, str(d), fails], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    # refused with nothing launched; then, with nothing failing, the whole call (from a thread without a context)
    assert json.loads(r.stdout) == [-4, 0, 0, launches]
