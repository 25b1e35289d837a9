"""Distributed shared memory may be touched only once every block of a cluster has started, which
the cluster's barrier shows and nothing else: in the source of each kernel that maps other blocks'
shared memory, a wait at that barrier stands in front of the first access."""
import os
import re

import pytest

from grouped_gemm_serving_gb300.build import CSRC

WAIT = re.compile(r"\b(?:cluster\.(?:sync|barrier_wait)|moe::cluster_sync)\(")
ACCESS = re.compile(r"\*\s*remote\(|\(remote\(")


def kernels():
    """(file, body) of the kernels that define `remote`, this tree's name for another block's copy of a variable."""
    out = []
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
            out += [(name, body) for body in re.split(r"\b__global__\b", text)[1:] if "map_shared_rank" in body]
    return out


def test_there_are_such_kernels():
    assert any(name == "sample.cu" for name, _ in kernels())


@pytest.mark.parametrize("name,body", [pytest.param(*k, id=k[0]) for k in kernels()])
def test_a_wait_stands_in_front(name, body):
    assert "remote = " in body, f"{name}: accesses of another block's memory go through `remote`"
    first, wait = ACCESS.search(body), WAIT.search(body)
    assert first and wait and wait.start() < first.start(), f"{name}: another block's memory before the cluster has met"
