"""Refusals of the feed-forward block's calls, and calls that fail in their host set-up (no GPU, nothing launched)."""
import ctypes
import glob
import json
import os
import subprocess
import sys

import pytest
import torch

from bwd_tri_attn_gb300 import _build

FAKE = 0x10000  # a 16-byte aligned address that is never dereferenced: validation fails first
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def tb():
    from bwd_tri_attn_gb300 import binding
    _build.build()
    binding.load()
    return binding


def shape(tb, M=40, ldx=0, lddout=0, C=64, F=128, act=0, wgrad_fp32=0):
    return tb.FfnShape(M, ldx, lddout, C, F, act, wgrad_fp32)


FWD = ("x", "Wg", "Wu", "Wd", "out", "a", "u", "workspace")
BWD = ("x", "Wg", "Wu", "Wd", "a", "u", "dout", "dx", "dWg", "dWu", "dWd", "workspace")


def call(tb, names, s, nulls=(), ws=1 << 40, **at):
    fn = tb.load().tri_ffn_fwd if names is FWD else tb.load().tri_ffn_bwd
    return fn(s, *[None if n in nulls else ctypes.c_void_p(at.get(n, FAKE)) for n in names], ctypes.c_size_t(ws), None)


@pytest.mark.parametrize("names", [FWD, BWD], ids=["fwd", "bwd"])
@pytest.mark.parametrize("bad,code", [(dict(M=0), -1), (dict(M=-1), -1), (dict(C=0), -1), (dict(F=-8), -1), (dict(act=3), -1),
                                      (dict(act=-1), -1), (dict(ldx=56), -1), (dict(lddout=-64), -1), (dict(C=60), -2),
                                      (dict(F=132), -2), (dict(M=(1 << 24) + 1), -2), (dict(C=(1 << 20) + 8), -2),
                                      (dict(F=(1 << 20) + 8), -2), (dict(ldx=68), -2), (dict(lddout=1 << 38), -2)])
def test_bad_shapes(tb, names, bad, code):
    s = shape(tb, **bad)
    assert call(tb, names, s) == code
    assert tb.tri_ffn_fwd_workspace_size(s) == tb.tri_ffn_bwd_workspace_size(s) == 0


def test_pointers(tb):
    s = shape(tb)
    for n in ("x", "Wg", "Wu", "Wd", "a", "u"):
        assert call(tb, FWD, s, nulls=(n,)) == -1
    assert call(tb, FWD, s, nulls=("out", "a", "u")) == -1
    for n in ("x", "Wg", "Wu", "Wd", "a", "u", "dout", "dWg", "dWu", "dWd"):
        assert call(tb, BWD, s, nulls=(n,)) == -1
    assert call(tb, BWD, s, nulls=("dx", "dWg", "dWu", "dWd")) == -1
    for names in (FWD, BWD):
        for n in names:
            assert call(tb, names, s, **{n: FAKE + 8}) == -2


def test_workspaces(tb):
    s = shape(tb)
    for names, need in ((FWD, tb.tri_ffn_fwd_workspace_size(s)), (BWD, tb.tri_ffn_bwd_workspace_size(s))):
        assert need > 0 and call(tb, names, s, ws=need - 1) == -3 and call(tb, names, s, nulls=("workspace",)) == -3


def test_binding_refuses_before_the_library(tb):
    bf = torch.bfloat16
    x, wg, wd = torch.zeros(4, 64, dtype=bf), torch.zeros(128, 64, dtype=bf), torch.zeros(64, 128, dtype=bf)
    fwd, bwd = tb.ffn_forward, tb.ffn_backward
    a = torch.zeros(4, 128, dtype=bf)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fwd(x, wg, wg, wd)
    with pytest.raises(ValueError, match="act must be"):
        fwd(x, wg, wg, wd, act="relu")
    with pytest.raises(ValueError, match="keep must be"):
        fwd(x, wg, wg, wd, keep="a")
    with pytest.raises(TypeError, match="Wu must be"):
        fwd(x, wg, wg.float(), wd)
    with pytest.raises(TypeError, match="x must be"):
        fwd(x.half(), wg, wg, wd)
    with pytest.raises(TypeError, match="Wd must be a torch.Tensor"):
        fwd(x, wg, wg, None)
    with pytest.raises(ValueError, match="Wg must have shape"):
        fwd(x, wd, wd, wg)
    with pytest.raises(ValueError, match="Wu must have shape"):
        fwd(x, wg, wg[:64], wd)
    with pytest.raises(ValueError, match="Wd must have shape"):
        fwd(x, wg, wg, wg)
    with pytest.raises(ValueError, match="Wg must be contiguous"):
        fwd(x, wd.t(), wg, wd)
    with pytest.raises(ValueError, match="at least one"):
        fwd(x[:0], wg, wg, wd)
    with pytest.raises(ValueError, match="evenly spaced"):
        fwd(x[:1].expand(4, 64), wg, wg, wd)
    with pytest.raises(ValueError, match="dout"):
        bwd(x, wg, wg, wd, a, a, x[:3])
    with pytest.raises(ValueError, match="a has"):
        bwd(x, wg, wg, wd, a[:3], a, x)
    with pytest.raises(TypeError, match="weight_dtype"):
        bwd(x, wg, wg, wd, a, a, x, weight_dtype=torch.float16)
    with pytest.raises(ValueError, match="no gradient"):
        bwd(x, wg, wg, wd, a, a, x, need_dx=False, need_dw=False)


def test_axes_that_32_bits_do_not_hold(tb):
    def meta(*s):
        return torch.empty(s, dtype=torch.bfloat16, device="meta")

    with pytest.raises(ValueError, match="too long"):
        tb.ffn_forward(meta(1, 2 ** 32 + 64), meta(8, 2 ** 32 + 64), meta(8, 2 ** 32 + 64), meta(2 ** 32 + 64, 8))
    with pytest.raises(ValueError, match="too long"):
        tb.ffn_forward(meta(1, 8), meta(2 ** 32 + 64, 8), meta(2 ** 32 + 64, 8), meta(8, 2 ** 32 + 64))


# Calls that fail in their set-up have enqueued nothing: the library's objects against a stand-in for the CUDA runtime that
# counts launches and fails the call it is told to, each case in a process of its own.
CHILD = """
import ctypes, json, sys
path, name, M, C, F, fails = sys.argv[1:]
class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("M", "ldx", "lddout")] + [(n, ctypes.c_int) for n in ("C", "F", "act", "f32")]
lib = ctypes.CDLL(path)
pointers = {"tri_ffn_fwd": 8, "tri_ffn_bwd": 12}[name]
call = getattr(lib, name)
call.argtypes = [Shape] + [ctypes.c_void_p] * pointers + [ctypes.c_size_t, ctypes.c_void_p]
seen = []
for f in (fails, ""):
    lib.fake_fail(f.encode())
    seen += [call(Shape(int(M), 0, 0, int(C), int(F), 0, 0), *[0x10000] * pointers, 1 << 40, None), lib.fake_launches()]
print(json.dumps(seen))
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    _build.build()
    objects = [os.path.join(_build.OBJDIR, os.path.basename(s)[:-3] + ".o") for s in glob.glob(os.path.join(_build.CSRC, "*.cu"))]
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    out = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-I", include, "-o", out, *objects, os.path.join(HERE, "csrc", "fake_runtime.cpp")],
                   check=True, capture_output=True)
    return out


@pytest.mark.parametrize("name,M,C,F,launches", [("tri_ffn_fwd", 1000, 512, 1024, 2), ("tri_ffn_fwd", 40000, 128, 512, 1),
                                                 ("tri_ffn_bwd", 1000, 512, 1024, 3)])
@pytest.mark.parametrize("fails", ["cudaFuncSetAttribute", "cuTensorMapEncodeTiled", "cudaGetSymbolAddress", "cudaGetDevice",
                                   "cudaDeviceGetAttribute", "cudaSetDevice"])
def test_nothing_is_enqueued(fake, name, M, C, F, launches, fails):
    r = subprocess.run([sys.executable, "-c", CHILD, fake, name, str(M), str(C), str(F), fails], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    assert json.loads(r.stdout) == [-4, 0, 0, launches]
