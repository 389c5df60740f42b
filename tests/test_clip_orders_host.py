"""Gradients whose axes lie in another order, as the clipping's calls see them (no GPU, nothing launched)."""
import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb


@pytest.fixture(autouse=True)
def cpu_tensors(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (a CPU tensor's)


def shapes():
    t = torch.zeros(2, 3, 4, 5)
    return [t[0, 0].t(), t.permute(3, 1, 0, 2), t.contiguous(memory_format=torch.channels_last),
            torch.zeros(1, 7, 1).permute(2, 1, 0), torch.zeros(5).as_strided((1, 5), (77, 1)), torch.zeros(3, 0).t()]


@pytest.mark.parametrize("i", range(6))
def test_any_order(i):
    g = shapes()[i]
    for out in (None, [torch.empty_like(g)]):
        rows, n, _ = tb._clip_array([g], out, written=True)
        assert n == (g.numel() > 0) and (not n or (rows[0], rows[2]) == (g.data_ptr(), g.numel()))


def test_refused():
    t = torch.zeros(6, 8)
    four = torch.zeros(2, 3, 4, 5)
    for bad in (four[:, :1].reshape(2, 1, 20).transpose(1, 2), t[:, :4], t[::2], t.t()[:3], t.expand(2, 6, 8), torch.zeros(4).expand(3, 4).t(),
                t.as_strided((4, 4), (1, 1))):
        with pytest.raises(ValueError, match="gradient 1 must be contiguous"):
            tb._clip_array([t, bad], None, written=False)
        with pytest.raises(ValueError, match="out 0 must be contiguous"):
            tb._clip_array([torch.zeros(bad.shape)], [bad], written=True)
    for g, out in ((t, torch.zeros(8, 6).t()), (t.t(), torch.zeros(8, 6)), (t.t(), torch.zeros(6, 8)),
                   (torch.zeros(2, 3, 4).permute(2, 0, 1), torch.zeros(2, 3, 4).permute(2, 1, 0))):
        with pytest.raises(ValueError, match="out 0 must have gradient 0's shape and strides"):
            tb._clip_array([g], [out], written=True)
    assert tb._clip_array([t], [torch.zeros(48)], written=True)[1] == 1  # (both in their own order: the shape does not matter)
