"""Kernels that may begin while the stream's kernel before still writes (launch_after) read by ordinary loads: the
non-coherent ones (__ldg, ld_stream, and what the compiler makes of const __restrict__ parameters) are for memory that nobody writes from
the reading kernel's start on, and no wait inside the kernel changes that."""
import glob
import os
import re

from bwd_tri_attn_gb300 import _build

# What such a kernel may read that way: it was complete before the kernel that its call begins with (launched in the ordinary
# way) started.
COMPLETE = {
    "cross_dkv_kernel": ["a.mask"],
    "cross_dq_kernel": ["a.mask", "a.nl", "a.nd"],  # (the preparation's, whose end the kernel between has waited for)
}
# Files all of whose kernels are launched so, with the functions that these call.
WHOLE = ("ffn.cuh", "ffn_fwd.cu", "ffn_bwd.cu", "ffn_few.cu", "ffn_block.cu", "norm_bwd.cuh", "clip.cu")


def sources():
    return {os.path.basename(p): open(p).read() for p in glob.glob(os.path.join(_build.CSRC, "*.cu*"))}


def dependent_kernels(text):
    return {re.sub(r"<.*", "", k) for k in re.findall(r"\blaunch_after\(\s*(\w+(?:<[^(]*?>)?)\s*,", text)}


def kernel(text, name):
    """A kernel's parameters and body (which ends with a brace at the line's start)."""
    at = re.search(r"__global__[^;{]*?\b" + name + r"\(", text)
    body = text.index(") {\n", at.end())
    return text[at.end():body], text[body:text.index("\n}\n", body)]


def test_reads_of_what_the_kernel_before_wrote():
    files = sources()
    seen = set()
    for text in files.values():
        for name in dependent_kernels(text):
            home = next(t for t in files.values() if re.search(r"__global__[^;{]*?\b" + name + r"\(", t))
            parameters, body = kernel(home, name)
            assert not re.search(r"\bconst\s+\w+\s*\*\s*__restrict__", parameters), name
            assert "wait_previous_kernel()" in body, name
            for read in re.findall(r"\b(?:__ldg|ld_stream)\(([^;]*)", body):
                assert any(read.startswith(c) for c in COMPLETE.get(name, [])), (name, read)
            seen.add(name)
    assert {"product_kernel", "join_kernel", "few_kernel", "block_kernel", "norm_kernel", "clip_kernel", "norm_reduce_kernel",
            "relpos_bwd_kernel", "relpos_reduce_kernel", "cross_dkv_kernel", "cross_dq_kernel", "cross_join_kernel",
            "cross_fwd_join_kernel"} <= seen
    for name in WHOLE:
        assert not re.search(r"\b(?:__ldg|ld_stream)\(", files[name]), name
