"""Memory of the allocating helpers' calls on a stream that is not the caller's current one, in both directions:
what the caller's stream has given back but still uses is not what such a call writes, and the results of one
stay as they are until the caller's stream is done with them. (What a call itself drops while its stream has yet to
run it is in test_cross_layer_gpu.py.)"""
import pytest
import torch

from bwd_tri_attn_gb300 import binding as tb
from bwd_tri_attn_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

MS10 = 20_000_000  # cycles: about 10 ms


def _normal(shape, seed, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _calls(seed):
    """Every allocating helper on inputs of this seed, as call(stream)."""
    q, do = (_normal((2, 300, 4, 64), seed + i) for i in (0, 1))
    k, v = (_normal((2, 600, 4, 64), seed + i) for i in (2, 3))
    x, g, dy = _normal((600, 256), seed + 4, torch.float32), torch.ones(256, device="cuda"), _normal((600, 256), seed + 5, torch.float32)
    a = {n: t.cuda() for n, t in wl.make_inputs(B=1, S=40, N=128, H=4, d=32, seed=seed, mask=("random", 0.05)).items()}
    p = [_normal((1, 128, 128, 32), seed + i) for i in range(6, 10)]
    m = {n: t.cuda() for n, t in wl.make_module_inputs(1, 64, 128, 4, 32, seed=seed, mask=("tail", 3)).items()}
    z = [m[n] for n in ("z", "gamma", "beta", "W", "wb", "Wo", "mask")]
    core = [a[n] for n in ("Q", "K", "V", "bias", "mask")]
    O, LSE = tb.cross_forward(q, k, v)
    _, mean, rstd = tb.norm_forward(x, g, g)
    kept = tb.checkpoint_pack(x)
    Oa, La, Ra = tb.forward(*core)
    X, A, Bm = tb.mul_forward(*p)
    _, saved = tb.module_forward(*z, 4, 32)
    ws = torch.empty(tb.tri_cross_bwd_workspace_size(tb.cross_shape_of(q, k, v)), dtype=torch.uint8, device="cuda")
    return {
        "cross_forward": lambda s: tb.cross_forward(q, k, v, stream=s),
        "cross_backward": lambda s: tb.cross_backward(q, k, v, O, LSE, do, stream=s),
        "cross_backward_workspace": lambda s: tb.cross_backward(q, k, v, O, LSE, do, workspace=ws, stream=s),
        "norm_forward": lambda s: tb.norm_forward(x, g, g, stream=s),
        "norm_forward_checkpoint": lambda s: (lambda r: (*r[:3], *r[3]))(tb.norm_forward(x, g, g, checkpoint=True, stream=s)),
        "norm_backward": lambda s: tb.norm_backward(x, g, mean, rstd, dy, stream=s),
        "norm_backward_no_weights": lambda s: tb.norm_backward(x, None, mean, rstd, dy, stream=s)[:1],
        "checkpoint_pack": lambda s: tuple(tb.checkpoint_pack(x, stream=s)),
        "checkpoint_unpack": lambda s: (tb.checkpoint_unpack(kept, torch.float32, stream=s),),
        "forward": lambda s: tb.forward(*core, stream=s),
        "backward": lambda s: tb.backward(*core, Oa, Ra, La, a["dO"], stream=s),
        "mul_forward": lambda s: tb.mul_forward(*p, stream=s),
        "mul_backward": lambda s: tb.mul_backward(*p, A, Bm, X, stream=s),
        "module_forward": lambda s: tb.module_forward(*z, 4, 32, stream=s)[:1],
        "module_backward": lambda s: tb.module_backward(*z, saved, m["dout"], 4, 32, stream=s),
    }


NAMES = ["cross_forward", "cross_backward", "cross_backward_workspace", "norm_forward", "norm_forward_checkpoint",
         "norm_backward", "norm_backward_no_weights", "checkpoint_pack", "checkpoint_unpack", "forward", "backward", "mul_forward",
         "mul_backward", "module_forward", "module_backward"]


@pytest.fixture(scope="module")
def calls():
    both = [_calls(100), _calls(200)]
    assert sorted(both[0]) == sorted(NAMES)
    torch.cuda.synchronize()
    return both


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_callers_stream_still_uses(calls, name, handle):
    """Fills of temporaries wait behind a pause of the caller's stream and their memory is given back at once; a call
    on another stream, which waits for nothing, must not be written over by them."""
    call, side = calls[0][name], torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    sizes = [t.numel() * t.element_size() for t in want] + [1 << n for n in range(9, 25)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(MS10)
    for n in sizes:
        torch.full((n,), 7, dtype=torch.uint8, device="cuda")
    got = call(side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert tb.tri_attn_device_status() == 0


@pytest.mark.parametrize("name", NAMES)
def test_results_that_the_callers_stream_still_reads(calls, name):
    """Results are read by the caller's stream after a pause and dropped at once; the next call on their stream, with
    other inputs, must not write over them."""
    side = torch.cuda.Stream()
    want = [t.clone() for t in calls[0][name](None)]
    torch.cuda.synchronize()
    got = calls[0][name](side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(MS10)
    copies = [t.clone() for t in got]
    del got
    later = [calls[1][name](side) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))
    assert len(later) == 3 and tb.tri_attn_device_status() == 0


def test_the_default_stream_by_its_handles():
    """From a side stream, 0 and cudaStreamLegacy are the default stream; cudaStreamPerThread is refused."""
    x = _normal((600, 256), 1)
    want = tb.norm_forward(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = [tb.norm_forward(x, stream=h) for h in (0, 1, torch.cuda.default_stream())]
        with pytest.raises(ValueError, match="per-thread"):
            tb.norm_forward(x, stream=2)
    got.append(tb.norm_forward(x, stream=1))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


def test_a_call_on_a_forked_stream_in_a_captured_graph():
    x, g, dy = _normal((600, 256), 2), torch.ones(256, device="cuda"), _normal((600, 256), 3)
    side = torch.cuda.Stream()

    def step(s):
        y, mean, rstd, kept = tb.norm_forward(x, g, g, checkpoint=True, stream=s)
        return (y, mean, rstd, *kept, *tb.norm_backward(kept, g, mean, rstd, dy, stream=s))

    want = step(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = step(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
