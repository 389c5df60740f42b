"""Gradients that share memory, as the clipping's calls see them (no GPU, nothing launched)."""
import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb


@pytest.fixture(autouse=True)
def cpu_tensors(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (a CPU tensor's)


def test_the_norm_takes_a_tensor_twice():
    g = torch.zeros(4, 4)
    rows, n, _ = tb._clip_array([g, g, g[1:]], None, written=False)
    assert n == 3 and list(rows[0::4]) == [g.data_ptr(), g.data_ptr(), g[1].data_ptr()] and list(rows[2::4]) == [16, 16, 12]
    with pytest.raises(ValueError, match="stands twice"):
        tb._clip_array([g, g], None, written=True)
