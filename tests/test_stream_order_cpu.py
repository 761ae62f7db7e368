"""Kernels that may be launched while the kernel before them in the stream runs:
each waits for it before it takes anything that a kernel in front may need, or
touches global memory.  Read from the sources: a GPU shows a breach only as a
hang."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_state_linear_gb300", "csrc")


def kernels(name):
    """(name, body) of every __global__ function of a source file, comments taken out."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for part in src.split("__global__")[1:]:
        head, rest = part.split(") {", 1)            # the end of the parameters
        depth, i = 1, 0
        while depth:
            depth += {"{": 1, "}": -1}.get(rest[i], 0)
            i += 1
        yield re.search(r"(\w+_kernel)\(", head).group(1), rest[:i]


@pytest.mark.parametrize("name", ["recurrence.cu", "residual_norm.cu"])
def test_waits_for_the_stream_first(name):
    found = list(kernels(name))
    assert len(found) >= 3
    for kernel, body in found:
        at = body.find("wait_for_stream()")
        assert at >= 0, kernel
        before = body[:at]
        for taken in ("tmem_alloc", "__ldg", "offsets_ok", "next_ticket", "record_status", "tma_load"):
            assert taken not in before, (kernel, taken)
