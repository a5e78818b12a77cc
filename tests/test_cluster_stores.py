"""A block of a cluster may touch another block's shared memory only once that
block has started: every kernel that does passes a cluster barrier first (checked
in the sources, since a GPU nearly always starts the blocks together)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_ffn_sort_b200",
                    "csrc")
REMOTE = re.compile(r"cluster_map_shared\(|st_cluster_v4\(|(?:st|ld|atom|red)\.shared::cluster")
WAIT = re.compile(r"cluster_(?:sync_all|wait)\(\)")


def kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for start in (m.start() for m in re.finditer("__global__", text)):
            body = text.index("{", start)
            depth = 0
            for end in range(body, len(text)):
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                if depth == 0:
                    break
            yield os.path.basename(path), text[body:end]


def first(pattern, text):
    m = pattern.search(text)
    return m.start() if m else None


REMOTE_KERNELS = [(name, body) for name, body in kernels() if REMOTE.search(body)]


def test_kernels_were_found():
    assert {name for name, _ in REMOTE_KERNELS} == {"grad_clip.cu", "router.cu"}


@pytest.mark.parametrize("name,body", REMOTE_KERNELS, ids=[n for n, _ in REMOTE_KERNELS])
def test_a_barrier_before_the_first_remote_access(name, body):
    at = first(WAIT, body)
    assert at is not None and at < first(REMOTE, body)
    # Either half of a split barrier is of use only with the other.
    assert body.count("cluster_arrive()") == body.count("cluster_wait()")
    if "cluster_wait()" in body:
        assert body.index("cluster_arrive()") < body.index("cluster_wait()")
    # No block leaves while others may still write to it.
    last = max(m.start() for m in REMOTE.finditer(body))
    assert WAIT.search(body, last)
