"""Refusals of the gradients' clipping and of the relative position bias, and its buckets (no GPU, nothing launched)."""
import ctypes
import math

import pytest
import torch

FAKE = 0x10000  # a 16-byte aligned address that is never dereferenced: validation fails first


@pytest.fixture(scope="module")
def tb():
    from bwd_tri_attn_gb300 import _build, binding
    _build.build()
    binding.load()
    return binding


def clip(tb, rows, max_norm=1.0, norm=FAKE, ws=FAKE, nbytes=16384, count=None):
    a = (tb.ClipTensor * max(len(rows), 1))(*rows)
    lib, n = tb.load(), len(rows) if count is None else count
    got = {lib.tri_clip(n, a, max_norm, norm, ws, nbytes, None)}
    if math.isfinite(max_norm) and max_norm >= 0 and all(r[1] for r in rows):
        got.add(lib.tri_grad_norm(n, a, norm, ws, nbytes, None))
    assert len(got) == 1
    return got.pop()


def test_clip(tb):
    good = (FAKE, FAKE, 100, 0)
    assert clip(tb, [good], max_norm=-1.0) == -1 and clip(tb, [good], max_norm=float("nan")) == -1
    assert clip(tb, [good], norm=None) == -1 and clip(tb, [good], count=-1) == -1
    assert clip(tb, [good, (FAKE, FAKE, 100, 3)]) == -1 and clip(tb, [(FAKE, FAKE, -1, 0)]) == -1
    assert clip(tb, [(None, FAKE, 1, 0)]) == -1 and clip(tb, [(FAKE, None, 1, 0)]) == -1
    assert clip(tb, [good], count=(1 << 20) + 1) == -2 and clip(tb, [(FAKE, FAKE, 1 << 47, 0)]) == -2
    assert clip(tb, [(FAKE + 1, FAKE, 9, 0)]) == -2 and clip(tb, [(FAKE + 2, FAKE, 9, 2)]) == -2
    assert tb.load().tri_clip(1, (tb.ClipTensor * 1)((FAKE, FAKE + 1, 9, 0)), 1.0, FAKE, FAKE, 16384, None) == -2
    assert clip(tb, [good], norm=FAKE + 2) == -2 and clip(tb, [good], ws=FAKE + 8) == -2
    assert clip(tb, [good], nbytes=16383) == -3 and clip(tb, [good], ws=None) == -3


def test_clip_binding(tb, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    g = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="gradient 0 must be a CUDA tensor"):
        tb.clip_gradients([g], 1.0)
    with pytest.raises(ValueError, match="max_norm"):
        tb.clip_gradients([g], -1.0)
    with pytest.raises(ValueError, match="max_norm"):
        tb.clip_gradients([g], float("nan"))
    with pytest.raises(ValueError, match="1 outputs for 2"):
        tb.clip_gradients([g, g], 1.0, out=[g])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (a CPU tensor's)
    with pytest.raises(TypeError, match="gradient 0 must be bfloat16"):
        tb.gradient_norm([g.double()])
    with pytest.raises(TypeError, match="gradient 1 must be a torch.Tensor"):
        tb.gradient_norm([g, 1.0])
    with pytest.raises(ValueError, match="gradient 0 must be contiguous"):
        tb.gradient_norm([g.t()[:2]])
    with pytest.raises(ValueError, match="out 0 must be a tensor of"):
        tb.clip_gradients([g], 1.0, out=[g[:3]])
    with pytest.raises(ValueError, match="out 0 must be a tensor of"):
        tb.clip_gradients([g], 1.0, out=[g.half()])
    with pytest.raises(ValueError, match="stands twice"):
        tb.clip_gradients([g, g], 1.0)
    with pytest.raises(ValueError, match="stands twice"):
        tb.clip_gradients([g, g.clone()], 1.0, out=[g, g])


STARTS = (0, 1, 2, 4)


def relpos(tb, s, starts=STARTS, fwd=(), bwd=(), ws=1 << 40, which=3, **at):
    arr = None if starts is None else (ctypes.c_int32 * max(len(starts), 1))(*starts)
    lib, got = tb.load(), set()
    if which & 1:
        names = ("table", "positions", "key_positions", "base", "bias")
        got.add(lib.tri_relpos_fwd(s, arr, *[None if n in fwd else at.get(n, FAKE) for n in names], None))
    if which & 2:
        names = ("positions", "key_positions", "dbias", "dtable", "workspace")
        got.add(lib.tri_relpos_bwd(s, arr, *[None if n in bwd else at.get(n, FAKE) for n in names], ws, None))
    assert len(got) == 1
    return got.pop()


def test_relpos(tb):
    def shape(B=1, H=2, Nq=5, Nk=7, K=4, two=1):
        return tb.RelposShape(B, H, Nq, Nk, K, two)

    for bad in (dict(B=0), dict(H=0), dict(Nq=-1), dict(Nk=0), dict(K=0), dict(two=2)):
        assert relpos(tb, shape(**bad)) == -1 and tb.tri_relpos_bwd_workspace_size(shape(**bad)) == 0
    for bad in (dict(K=129), dict(B=1025, H=1024), dict(Nq=1 << 16, Nk=1 << 15), dict(Nq=1, Nk=1 << 30)):
        assert relpos(tb, shape(**bad)) == -2 and tb.tri_relpos_bwd_workspace_size(shape(**bad)) == 0
    for starts in (None, (1, 2, 3, 4), (0, 2, 2, 3), (0, 3, 2, 5), (0, 1, 2, -4)):
        assert relpos(tb, shape(), starts) == -1
    for n in ("table", "bias", "positions", "key_positions"):
        assert relpos(tb, shape(), fwd=(n,), which=1) == -1
    for n in ("dbias", "dtable", "positions", "key_positions"):
        assert relpos(tb, shape(), bwd=(n,), which=2) == -1
    for n, off in (("table", 2), ("bias", 8), ("base", 2), ("positions", 1), ("key_positions", 2)):
        assert relpos(tb, shape(), which=1, **{n: FAKE + off}) == -2
    for n, off in (("dbias", 8), ("dtable", 2), ("workspace", 2)):
        assert relpos(tb, shape(), which=2, **{n: FAKE + off}) == -2
    need = tb.tri_relpos_bwd_workspace_size(shape())
    assert need and relpos(tb, shape(), which=2, ws=need - 1) == -3 and relpos(tb, shape(), which=2, bwd=("workspace",)) == -3


def test_relpos_long_planes_are_split(tb):
    """However many planes there are, a lane (of 128 of a CTA) adds up at most 2^14 values in one FP32 sum: every CTA of a
    plane has its own row of partial sums in the workspace."""
    for B, H, Nq, Nk in ((152, 7, 4096, 4096), (1 << 17, 7, 2048, 2048), (1, 1, 46340, 46340), (152, 6, 1 << 16, 32767)):
        need = tb.tri_relpos_bwd_workspace_size(tb.RelposShape(B, H, Nq, Nk, 4, 1))
        ctas = need // (4 * 8 * B * H)
        assert ctas * 128 * (1 << 14) >= Nq * Nk, (B, H, Nq, Nk)


def test_relpos_binding(tb):
    t, starts = torch.zeros(8, 2), STARTS
    d = torch.zeros(1, 2, 5, 7, dtype=torch.bfloat16)
    pos = torch.zeros(1, 5, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tb.relpos_forward(t, starts, 5, 7)
    with pytest.raises(ValueError, match="table must have shape"):
        tb.relpos_forward(t, starts, 5, 7, two_sided=False)
    with pytest.raises(TypeError, match="table must be"):
        tb.relpos_forward(t.half(), starts, 5, 7)
    for bad in ((), (1, 2), (0, 2, 1), (0, 0), (0, 1 << 31)):
        with pytest.raises(ValueError, match="starts"):
            tb.relpos_forward(torch.zeros(2 * len(bad), 2), bad, 5, 7)
    with pytest.raises(ValueError, match="base has shape"):
        tb.relpos_forward(t, starts, 5, 6, base=d)
    with pytest.raises(ValueError, match="keys need positions"):
        tb.relpos_forward(t, starts, 5, 7, positions=pos)
    with pytest.raises(ValueError, match="come with positions"):
        tb.relpos_forward(t, starts, 5, 7, key_positions=pos)
    with pytest.raises(ValueError, match="positions has shape"):
        tb.relpos_forward(t, starts, 5, B=2, positions=pos)
    with pytest.raises(TypeError, match="positions must be"):
        tb.relpos_forward(t, starts, 5, positions=pos.long())
    with pytest.raises(ValueError, match="too long"):
        tb.relpos_forward(t, starts, 2 ** 32 + 1)
    with pytest.raises(ValueError, match="four axes"):
        tb.relpos_backward(d[0], starts)
    with pytest.raises(TypeError, match="dbias must be"):
        tb.relpos_backward(d.float(), starts)
    with pytest.raises(ValueError, match="dbias must be contiguous"):
        tb.relpos_backward(d.transpose(2, 3), starts)


def test_logarithmic_buckets(tb):
    """Against the definition in whole numbers, and the usual table of 32 buckets to 128."""
    assert tb.relpos_starts(32, 128) == (0, 1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 23, 32, 46, 64, 91)
    assert tb.relpos_starts(2, 1) == (0,) and tb.relpos_starts(1, 5, two_sided=False) == (0,)
    for K in (1, 2, 3, 5, 8, 16, 33, 64):
        for far in (K, K + 1, 3 * K, 100 * K):
            s = tb.relpos_starts(K, far, two_sided=False)
            e = (K + 1) // 2
            assert len(s) == K and s[:e] == tuple(range(e)) and all(b > a for a, b in zip(s, s[1:]))
            for k in range(K - e):
                n, m = s[e + k], K - e
                at_least = n ** m * e ** k >= far ** k * e ** m
                before = (n - 1) ** m * e ** k >= far ** k * e ** m
                assert at_least and (not before or n == s[e + k - 1] + 1)
    for bad in ((0, 5), (3, 5), (8, 3)):
        with pytest.raises(ValueError):
            tb.relpos_starts(*bad)
