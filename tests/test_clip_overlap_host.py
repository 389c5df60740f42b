"""Gradients that share memory, as the clipping's calls see them (no GPU, nothing launched)."""
import glob
import json
import os
import random
import subprocess
import sys

import pytest
import torch

from bwd_tri_attn_gb300 import _build, binding as tb

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(autouse=True)
def cpu_tensors(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (a CPU tensor's)


def test_the_norm_takes_a_tensor_twice():
    g = torch.zeros(4, 4)
    rows, n, _ = tb._clip_array([g, g, g[1:]], None, written=False)
    assert n == 3 and list(rows[0::4]) == [g.data_ptr(), g.data_ptr(), g[1].data_ptr()] and list(rows[2::4]) == [16, 16, 12]
    with pytest.raises(ValueError, match="stands twice"):
        tb._clip_array([g, g], None, written=True)


# The library's objects against a stand-in for the CUDA runtime (launches are counted, none runs), in a process of its own: the
# addresses are no memory.
CHILD = """
import ctypes, json, sys
path, cases = sys.argv[1], json.loads(sys.argv[2])
class Tensor(ctypes.Structure):
    _fields_ = [(n, t) for n, t in zip(("g", "out", "n", "dtype"), (ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64))]
lib = ctypes.CDLL(path)
seen = []
for rows in cases:
    t = (Tensor * max(len(rows), 1))(*[tuple(r) for r in rows])
    before = lib.fake_launches()
    clip = lib.tri_clip(len(rows), t, ctypes.c_float(1.0), ctypes.c_void_p(1 << 40), ctypes.c_void_p(1 << 41), ctypes.c_size_t(1 << 20), None)
    launched = lib.fake_launches() - before
    norm = lib.tri_grad_norm(len(rows), t, ctypes.c_void_p(1 << 40), ctypes.c_void_p(1 << 41), ctypes.c_size_t(1 << 20), None)
    seen.append([clip, launched > 0, norm])
print(json.dumps(seen))
"""


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    _build.build()
    objects = [os.path.join(_build.OBJDIR, os.path.basename(s)[:-3] + ".o") for s in glob.glob(os.path.join(_build.CSRC, "*.cu"))]
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    out = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-I", include, "-o", out, *objects, os.path.join(HERE, "csrc", "fake_runtime.cpp")],
                   check=True, capture_output=True)

    def run(cases):
        r = subprocess.run([sys.executable, "-c", CHILD, out, json.dumps(cases)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        return json.loads(r.stdout)

    return run


A, B, C, D = (0x100000 * k for k in (1, 2, 3, 4))
F32, BF16 = 2, 0
APART = {
    "in place": [(A, A, 100, F32), (B, B, 100, F32)],
    "end to end": [(A, A, 100, F32), (A + 400, A + 400, 100, F32), (A + 800, A + 800, 7, BF16)],
    "into others": [(A, C, 100, F32), (B, D, 100, F32)],
    "one and the other": [(A, A, 100, F32), (B, D, 100, F32)],
    "read twice": [(A, C, 100, F32), (A, D, 100, F32), (A + 40, B, 100, F32)],
    "nothing": [],
    "without elements": [(A, A, 0, F32), (A, A, 100, F32), (A + 8, A + 8, 0, BF16)],
    "beside each other": [(A, A + 400, 100, F32), (B, B - 200, 100, BF16)],
    "many": [(A + 400 * k, A + 400 * k, 100, F32) for k in range(1000)],
    "many, into others": [(A + 400 * k, B + 400 * (999 - k), 100, F32) for k in range(1000)],
}
SHARED = {
    "twice in place": [(A, A, 100, F32), (A, A, 100, F32)],
    "one output twice": [(A, C, 100, F32), (B, C, 100, F32)],
    "swapped": [(A, B, 100, F32), (B, A, 100, F32)],
    "in a ring": [(A, B, 100, F32), (B, C, 100, F32), (C, A, 100, F32)],
    "an output that another one reads": [(A, B, 100, F32), (B, D, 100, F32)],
    "in place and read": [(A, A, 100, F32), (A, D, 100, F32)],
    "partly, in place": [(A, A, 100, F32), (A + 396, A + 396, 100, F32)],
    "partly, one input and its output": [(A, A + 16, 100, F32)],
    "partly, before": [(A, A - 2, 100, BF16)],
    "partly, outputs": [(A, C, 100, F32), (B, C + 398, 100, BF16)],
    "a long one over short ones": [(A, A, 1000, F32), (A + 2000, A + 2000, 1, BF16), (B, B, 1, F32)],
    "a long one read": [(A, C, 1000, F32), (D, A + 3996, 2, BF16)],
    "many": [(A + 400 * k, A + 400 * k - 4 * (k == 777), 100, F32) for k in range(1000)],
    "many, into others": [(A + 400 * k, B + 400 * (999 - k) - 4 * (k == 500), 100, F32) for k in range(1000)],
}


def test_what_is_written_lies_apart(calls):
    """The norm, which writes nothing there, takes them all."""
    got = calls(list(APART.values()) + list(SHARED.values()))
    for name, g in zip(list(APART), got):
        assert g == [0, True, 0], name
    for name, g in zip(list(SHARED), got[len(APART):]):
        assert g == [-1, False, 0], name


def test_against_every_pair(calls):
    """Random ranges, against the definition."""
    rng = random.Random(5)
    cases = [[(A + 4 * rng.randrange(120), rng.choice([0, A]) + 4 * rng.randrange(1, 120), rng.randrange(0, 9), F32)
              for _ in range(rng.randrange(1, 6))] for _ in range(400)]
    cases = [[(g, out if out > A else g, n, t) for g, out, n, t in rows] for rows in cases]

    def apart(rows):
        spans = [((g, g + 4 * n), (o, o + 4 * n)) for g, o, n, _ in rows if n]

        def meet(x, y):
            return x[0] < y[1] and y[0] < x[1]
        for i, (g, o) in enumerate(spans):
            if g != o and meet(g, o):
                return False
            if any(meet(o, other) for j, pair in enumerate(spans) if j != i for other in pair):
                return False
        return True

    got = calls(cases)
    assert {c for c, _, _ in got} == {0, -1}
    for rows, (clip, launched, norm) in zip(cases, got):
        assert (clip, launched, norm) == ((0, True, 0) if apart(rows) else (-1, False, 0)), rows
