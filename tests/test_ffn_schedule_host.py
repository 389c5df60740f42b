"""The waits of the feed-forward block's one-kernel forward, in a model on the host (tests/csrc/ffn_block_model.cpp): copies and
products may finish in any order that the hardware allows, and no wait may pass a phase early. The model takes its barriers
and phases from the header that the kernel takes them from."""
import os
import re
import subprocess

import pytest

from bwd_tri_attn_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("model") / "model")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", _build.CSRC, "-o", out, os.path.join(HERE, "csrc", "ffn_block_model.cpp")],
                   check=True, capture_output=True)

    def run(channels, shared, seed, runs=700):
        r = subprocess.run([out, *map(str, (channels, shared, seed, runs))], check=True, capture_output=True, text=True, timeout=120)
        return [int(x) for x in r.stdout.split()]

    return run


@pytest.mark.parametrize("seed", [0, 10 ** 6, 2 * 10 ** 6])
@pytest.mark.parametrize("channels", [128, 256])
def test_no_wait_passes_early(model, channels, seed):
    assert model(channels, 0, seed) == [0, 0, 0]  # early waits, runs that stood still, wrong numbers of arrivals


def test_the_model_sees_a_shared_barrier(model):
    """Three buffers with one barrier each, at which two groups of warps wait in turn: a group misses every second phase."""
    early, still, _ = model(128, 1, 0)
    assert early > 0 and still > 0


def test_the_kernel_has_the_models_buffers():
    with open(os.path.join(_build.CSRC, "ffn_block.cu")) as f:
        text = f.read()
    for line in ("NS = CB == 128 ? 3 : 2;", "NW = CB == 128 ? 5 : 3;", "XB = CB == 128 ? 2 : 1,", "using Order = BlockSchedule<NS, NW>;"):
        assert line in text
    waits = re.findall(r"C::B_(?:S|H|WF|WE) \+ (\w+(?:::\w+\(\w+\))?)", text)
    assert len(waits) >= 10 and all(w in ("b", "s") or w.startswith("Order::") for w in waits)
    assert re.findall(r"[bs] = (\w+::\w+)\((?:n|ws)\)", text) == ["Order::slot"] + ["Order::buffer", "Order::slot"] * 2 + ["Order::buffer"]
