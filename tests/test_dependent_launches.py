"""Kernels launched as programmatic dependents wait for the kernel before them
ahead of every return, read from the sources (no GPU).

Such a kernel may start before its predecessor is done, and what follows on
the stream is ordered after it alone: a grid whose blocks return without the
wait can end first, and the next reader of the predecessor's outputs is then
ordered after nothing."""
import os
import re

import pytest

from tree_speculative_decoding_attn_gb300 import _build


def kernels():
    """(file, name, body) of every kernel that waits for its predecessor."""
    for f in sorted(os.listdir(_build.CSRC)):
        if not f.endswith((".cu", ".cuh")):
            continue
        text = re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, f)).read())
        for m in re.finditer(r"__global__\s+void\s+(?:__\w+__\s*\([^()]*\)\s*)*(?!__)(\w+)\s*\(", text):
            end = text.find("\n}", m.end())
            body = text[text.index("{", m.end()):end]
            if "grid_dep_wait()" in body:
                yield f, m.group(1), body


FOUND = [k for k in kernels() if "pdl_wait" not in k[2]]  # (the GEMM's producers wait where they are told to)


def test_the_merge_and_copy_kernels_are_among_them():
    assert {"attn_tc2_combine_kernel", "attn_tc2_window_combine_kernel", "pages_copy_kernel"} <= {k[1] for k in FOUND}


@pytest.mark.parametrize("name,body", [k[1:] for k in FOUND], ids=[k[1] for k in FOUND])
def test_nothing_returns_before_the_wait(name, body):
    head = body[:body.rindex("grid_dep_wait()")]
    assert not re.search(r"\breturn\s*;", head), f"{name} returns before its wait"
