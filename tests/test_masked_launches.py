"""Rules that the kernels of ress_masked_attn keep where they overlap one another.

A kernel that is launched while the one before it still runs (griddepcontrol.wait) must not
read that one's results as read-only data: the read-only path assumes memory that nobody
writes for the kernel's whole life, so such a load may be moved above the wait or served from
a stale line.  Checked on the sources, since the hardware rarely shows it.
"""
import os
import re

from block_sparse_global_b200 import build as B


def _kernels(name):
    """{kernel: (parameters, body)} of a source file."""
    text = open(os.path.join(B.CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    out = {}
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^)]*\)\s*)?(\w+)\s*\(", text):
        at, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        params = text[m.end():at - 1]
        start = at = text.index("{", at) + 1
        depth = 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        out[m.group(1)] = (params, text[start:at - 1])
    return out


def test_overlapped_kernels_do_not_read_results_as_constants():
    kernels = {k: v for k, v in _kernels("k_masked_attn.cu").items() if "wait_prerequisites()" in v[1]}
    assert set(kernels) == {"masked_attn_kernel", "plan_kernel", "rank_kernel", "join_kernel"}
    for name, (params, body) in kernels.items():
        assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", params), name
        for arg in re.findall(r"__ldg\(\s*([^;]*)", body):    # the caller's arrays are written by nobody
            assert re.match(r"p\.[qk]_(doc|order|pos)\b", arg), (name, arg)
