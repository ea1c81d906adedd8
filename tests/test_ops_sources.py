"""What the kernels' sources have to keep that no run on one machine can show: the order of a
cluster's barrier and the stores into other blocks' shared memory."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "permute_grouped_gemm_gb300", "csrc")


def body_of(source, kernel):
    """The body of a kernel, comments left out."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, source)).read())
    start = text.index("{", re.search(r"\b%s\(" % kernel, text).end()) + 1
    depth, i = 1, start
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[start:i]


BARRIER = re.compile(r"\b(?:ptx::)?(?:cluster_sync|cluster_all_started)\(\)")
REMOTE = re.compile(r"\bst_cluster_\w+\(|\bmbar_arrive_remote\w*\(")


def first(pattern, body):
    m = pattern.search(body)
    return m.start() if m else None


@pytest.mark.parametrize("source,kernel,through", [
    ("adapters_few.cu", "few_shrink_kernel", None),
    ("ops_prep.cu", "adapter_prep_small_kernel", None),
    ("rows_skinny.cu", "rows_skinny_kernel", "epilogue<"),
    ("rows_outer.cu", "rows_outer_kernel", "epilogue<"),
    ("rows_wide.cu", "rows_wide_kernel", "w_producer<"),
])
def test_every_block_of_a_cluster_has_started_before_another_writes_to_it(source, kernel, through):
    body = body_of(source, kernel)
    barrier = first(BARRIER, body)
    # the first remote write, or the call of the function that makes it
    write = body.find(through) if through else first(REMOTE, body)
    assert write is not None and write >= 0
    assert barrier is not None and barrier < write
    if "cluster_all_started" in body[barrier:barrier + 40]:
        assert body.find("cluster_started();") in range(0, barrier)


def test_the_kernels_with_remote_writes_are_the_ones_looked_at():
    new = {"adapters_few.cu", "rows_skinny.cu", "rows_outer.cu", "ops_prep.cu"}
    have = {f for f in os.listdir(CSRC) if f.endswith(".cu")
            and re.search(r"\bst_cluster_[uf]32\(", open(os.path.join(CSRC, f)).read())}
    assert have == new
