"""The C ABI of LayerNorm, checkpoints and cross attention as declared, exported and bound (no GPU)."""
import glob
import os
import re

from bwd_tri_attn_gb300 import _build, binding as tb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _declared():
    names = set()
    for h in glob.glob(os.path.join(ROOT, "include", "*.h")):
        text = re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
        names |= set(re.findall(r"^(?:int|size_t|const char \*)\s*(tri_\w+)\(", text, flags=re.M))
    return names


def test_every_function_is_exported_and_bound():
    _build.build()
    lib = tb.load()
    names = _declared()
    assert names == set(tb.EXPORTS) and {"tri_norm_fwd", "tri_ckpt_pack", "tri_cross_bwd"} <= names
    for n in names:
        assert hasattr(lib, n) and getattr(lib, n).argtypes is not None, n


def test_error_texts_fit_every_operator():
    """The codes are shared: no text names one operator's sizes or functions."""
    for code in (-1, -2, -3):
        text = tb.strerror(code)
        assert text and not re.search(r"16 or 32|TRI_ATTN_MAX|tri_attn_bwd", text), text
