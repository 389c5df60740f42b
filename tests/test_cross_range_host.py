"""Scales whose product with log2(e), by which the kernels multiply scores, is no FP32 number (no GPU)."""
import pytest

from tests.test_cross_host import bwd, fwd, shape, tb  # noqa: F401 (tb: the fixture)


@pytest.mark.parametrize("scale", [2.5e38, -2.5e38, 3.4e38, -3.4e38])
def test_scale_too_large(tb, scale):  # noqa: F811
    s = shape(tb, scale=scale)
    assert fwd(tb, s) == -2 and bwd(tb, s) == -2
    assert tb.tri_cross_fwd_workspace_size(s) == 0 and tb.tri_cross_bwd_workspace_size(s) == 0
