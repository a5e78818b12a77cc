"""Kernels that are launched as programmatic dependents (launch_after.cuh) wait for what
runs before them before they read or write memory, and before any block leaves
(checked in the sources)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_ffn_sort_b200",
                    "csrc")
FILES = ["grad_clip.cu", "route_bwd.cu", "rows.cu"]


def kernels(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for start in (m.start() for m in re.finditer("__global__", text)):
        body = text.index("{", start)
        depth = 0
        for end in range(body, len(text)):
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            if depth == 0:
                break
        yield re.search(r"(\w+_kernel)\(", text[start:body]).group(1), text[body:end]


EVERY = [(name, kernel, body) for name in FILES for kernel, body in kernels(name)]


def test_these_are_the_files():
    users = {f for f in os.listdir(CSRC) if f.endswith(".cu") and "launch_after(" in open(os.path.join(CSRC, f)).read()}
    assert users == set(FILES) and len(EVERY) >= 12


@pytest.mark.parametrize("name,kernel,body", EVERY, ids=[k for _, k, _ in EVERY])
def test_the_wait_comes_first(name, kernel, body):
    before, wait, _ = body.partition("grid_dependency_wait();")
    assert wait, "no wait"
    assert not re.search(r"__ldg\(|\breturn\b|report_status|\bposition\(", before)
    # No value of a global array before the wait: only addresses of it are formed.
    for pointer in ("x", "inv", "w", "y_sorted", "y_shared", "dout", "ids", "dw", "logits", "zero_mask", "partial",
                    "sumsq", "n_rows"):
        assert not re.search(r"(?<![\w.>])%s\s*\[|\*\s*%s\b(?!\s*[\w*])" % (pointer, pointer), before), pointer
