"""Copies that the autograd glue makes of contiguous tensors (no GPU)."""
import torch

from bwd_tri_attn_gb300.autograd import _dense


def test_dense():
    t = torch.arange(64, dtype=torch.bfloat16)
    assert _dense(t) is t
    assert _dense(t[8:]).data_ptr() == t.data_ptr() + 16         # a view from a boundary on
    for part in (t[1:], t[4:12], t.view(8, 8).t(), t[::2]):
        c = _dense(part)
        assert c.is_contiguous() and c.data_ptr() % 16 == 0 and torch.equal(c, part)
