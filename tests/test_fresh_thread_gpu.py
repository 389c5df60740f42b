"""Calls from host threads that have made no CUDA call before (autograd's backward thread is one): a thread has no
current context then, and a call's first need of one may be a tensor map's. Every test is a process of its own, in
which another thread has done every one-time set-up and given memory back for the call to use."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import threading
import torch
from tests.test_streams_gpu import _calls
from bwd_tri_attn_gb300 import binding as tb
calls, out = _calls(100), {}
names = sorted(calls)
want = {n: [t.clone() for t in calls[n](None)] for n in names}
torch.cuda.synchronize()
def work(n):
    try:
        out[n] = calls[n](None)
    except Exception as e:
        out[n] = e
for n in names:
    t = threading.Thread(target=work, args=(n,))
    t.start()
    t.join()
    assert not isinstance(out[n], Exception), f"{n}: {out[n]}"
torch.cuda.synchronize()
for n in names:
    assert all(torch.equal(a, b) for a, b in zip(out[n], want[n])), n
assert tb.tri_attn_device_status() == 0
"""

BACKWARD = """
import torch
from bwd_tri_attn_gb300 import autograd as ag
gen = torch.Generator(device="cuda").manual_seed(1)
q, k, v = (torch.randn((2, n, 4, 64), generator=gen, device="cuda").bfloat16().requires_grad_() for n in (60, 130, 130))
p = [torch.randn((1, 40, 40, 24), generator=gen, device="cuda").bfloat16().requires_grad_() for _ in range(4)]
out, leaves = {"cross": (lambda: ag.cross_attention(q, k, v), [q, k, v]),
               "mul": (lambda: ag.triangle_multiplication(*p), p)}[WHICH]
O = out()
grads = torch.autograd.grad(O, leaves, torch.ones_like(O))  # (the backward thread's first work)
torch.cuda.synchronize()
assert all(g.isfinite().all() for g in grads)
"""


def _run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_every_call():
    _run(CHILD)


@pytest.mark.parametrize("which", ["cross", "mul"])
def test_backward_thread(which):
    _run(f"WHICH = {which!r}\n" + BACKWARD)
