"""The forward's workspace of few rows is the hidden features' room alone: a token asks for no room for tiles that several
SMs share (no GPU)."""
import pytest

from bwd_tri_attn_gb300 import _build, binding as tb


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    tb.load()


@pytest.mark.parametrize("M,C,F", [(1, 8, 8), (1, 4096, 16384), (16, 1 << 20, 1 << 20), (17, 1024, 4096), (32, 512, 8192)])
def test_few_rows(M, C, F):
    need = tb.tri_ffn_fwd_workspace_size(tb.FfnShape(M, 0, 0, C, F, 0, 0))
    assert 2 * M * F <= need < 2 * M * F + 256


@pytest.mark.parametrize("M,C,F", [(17, 4096, 16384), (32, 1032, 4096), (33, 8, 8), (147456, 128, 512)])
def test_tiles(M, C, F):
    """152 SMs: a pair of them has two shares of 256 x 256 FP32 sums at most."""
    assert tb.tri_ffn_fwd_workspace_size(tb.FfnShape(M, 0, 0, C, F, 0, 0)) >= 2 * M * F + 2 * 76 * 256 * 256 * 4
