"""Forward-mode derivatives: no operator of the library has them, and every one says so rather than return outputs
without a tangent, which reads as a derivative of zero (no GPU: the library's calls are replaced)."""
import types

import pytest
import torch
import torch.autograd.forward_ad as fwd_ad

from bwd_tri_attn_gb300 import autograd

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def stubs(monkeypatch):
    tb = autograd.tb

    def ffn_forward(x, Wg, Wu, Wd, act="silu", keep=False, **_):
        a = torch.zeros(*x.shape[:-1], Wg.shape[0], dtype=x.dtype)
        out = x.detach().clone()
        return (a, a) if keep == "only" else (out, a, a.clone()) if keep else out

    def rms_forward(x, gamma=None, residual=None, eps=1e-5, eight_bits=False, **_):
        y, rstd = x.detach().clone(), torch.zeros(x.shape[:-1])
        y8 = (torch.zeros(x.shape, dtype=torch.int8), rstd) if eight_bits else None
        return types.SimpleNamespace(y=y, rstd=rstd, r=None if residual is None else x.detach().clone(), y8=y8)

    monkeypatch.setattr(tb, "ffn_forward", ffn_forward)
    monkeypatch.setattr(tb, "rms_forward", rms_forward)
    monkeypatch.setattr(tb, "checkpoint_pack", lambda x: (torch.zeros(x.shape, dtype=torch.int8), torch.zeros(x.shape[0], 1)))
    monkeypatch.setattr(tb, "relpos_forward", lambda table, starts, Nq, *_: torch.zeros(1, table.shape[1], Nq, Nq, dtype=BF16))


C, F = 16, 24
SHAPES = {"x": (4, C), "residual": (4, C), "gamma": (C,), "Wg": (F, C), "Wu": (F, C), "Wd": (C, F)}


def arguments(names, dual, grad=()):
    made = {}
    for n in names:
        t = torch.randn(SHAPES[n]).to(BF16)
        if n in grad:
            t.requires_grad_()
        made[n] = fwd_ad.make_dual(t, torch.ones_like(t)) if n == dual else t
    return made


BLOCK, LAYER = ("x", "Wg", "Wu", "Wd"), ("x", "residual", "gamma", "Wg", "Wu", "Wd")
CALLS = [(autograd.gated_feed_forward, BLOCK, n) for n in BLOCK] + [(autograd.feed_forward_layer, LAYER, n) for n in LAYER]


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("grad", [False, True], ids=["no_grad", "grad"])
@pytest.mark.parametrize("call,names,dual", CALLS, ids=lambda v: getattr(v, "__name__", v if isinstance(v, str) else None))
def test_feed_forward(call, names, dual, grad, checkpoint):
    with torch.set_grad_enabled(grad), fwd_ad.dual_level():
        with pytest.raises(RuntimeError, match="jvp"):
            call(**arguments(names, dual), checkpoint=checkpoint)
        with pytest.raises(RuntimeError, match="jvp"):
            call(**arguments(names, dual, grad=names), checkpoint=checkpoint)
        got = call(**arguments(names, None), checkpoint=checkpoint)  # (inside a level, but without a tangent)
        assert all(fwd_ad.unpack_dual(t).tangent is None for t in (got if isinstance(got, tuple) else (got,)))


@pytest.mark.parametrize("grad", [False, True], ids=["no_grad", "grad"])
def test_module_with_frozen_weights(grad):
    layer = autograd.FeedForwardLayer(C, F).requires_grad_(False)
    x = torch.randn(4, C).to(BF16)
    with torch.set_grad_enabled(grad), fwd_ad.dual_level():
        with pytest.raises(RuntimeError, match="jvp"):
            layer(fwd_ad.make_dual(x, torch.ones_like(x)), x)


@pytest.mark.parametrize("grad", [False, True], ids=["no_grad", "grad"])
def test_the_others(grad):
    x, table = torch.randn(4, C).to(BF16), torch.randn(4, 2)
    with torch.set_grad_enabled(grad), fwd_ad.dual_level():
        with pytest.raises(RuntimeError, match="jvp"):
            autograd.rms_norm(fwd_ad.make_dual(x, torch.ones_like(x)))
        with pytest.raises(RuntimeError, match="jvp"):
            autograd.relative_position_bias(fwd_ad.make_dual(table, torch.ones_like(table)), (0, 1), 8)


def test_functional_transform():
    x, w = torch.randn(4, C).to(BF16), [torch.randn(SHAPES[n]).to(BF16) for n in ("Wg", "Wu", "Wd")]
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda t: autograd.gated_feed_forward(t, *w), (x,), (torch.ones_like(x),))
