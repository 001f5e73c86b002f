"""Every launch of the library is a programmatic dependent of the one before it
on the stream: it may start, and end, while that one still runs.  What orders
it is its own ``griddepcontrol.wait``; and the launch behind it, which waits for
it alone, relies on that for everything earlier.  So every thread that a kernel
lets go has to have passed the wait."""
import glob
import os
import re

import pytest

from decode_attention_paged_pa_gb300 import build

WAIT = "griddepcontrol.wait"


def bodies():
    """(file, kernel, body) of every __global__ function of the library."""
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__", text):
            at = text.index("{", m.end())
            name = re.findall(r"(\w+)\s*\(", text[m.end():at])
            depth, end = 0, at
            while True:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
                if depth == 0:
                    break
            yield os.path.basename(path), [n for n in name if n.endswith("kernel")][-1], text[at:end]


KERNELS = list(bodies())


def test_the_kernels_are_found():
    assert {k for _, k, _ in KERNELS} >= {"pa_clear_header_kernel", "pa_decode_kernel", "pa_combine_kernel",
                                          "pa_combine_rows_kernel", "kv4_decode_kernel", "kv4_tokens_kernel",
                                          "pages_plan_kernel", "pages_apply_kernel"}


@pytest.mark.parametrize("file,kernel,body", KERNELS, ids=[f"{f}:{k}" for f, k, _ in KERNELS])
def test_nothing_leaves_a_kernel_before_its_wait(file, kernel, body):
    assert WAIT in body
    before = body[:body.index(WAIT)]
    assert not re.search(r"\breturn\b", before), f"{file}: {kernel} may end before the launch it depends on"
    # (Not inside a branch either: the braces before it are closed, but for the body's own.)
    assert before.count("{") - before.count("}") == 1
