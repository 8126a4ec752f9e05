"""Host-only check of the kernels' sources: a block may touch the shared memory
of another block of its cluster only once that block is known to run, so every
kernel passes a cluster barrier before its first exchange with its peers.
(Nothing a run returns shows a missing barrier: the loads before the first
exchange nearly always take longer than the blocks' start.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_mixed_precision_scale_gb300",
                    "csrc")
# what reads or writes a peer's shared memory, or leaves an address of it behind
EXCHANGE = ("cluster_sum(", "mapa_shared(", "mbar_arrive_cluster(")


def kernels(path):
    """(name, body) of the __global__ functions of a source, comments blanked."""
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__global__", text):
        start = text.index("{", m.end())
        depth, end = 0, start
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield re.findall(r"(\w+)\s*\(", text[m.end():start])[-1], text[start:end]


@pytest.mark.parametrize("source", ["norm.cu", "gemm.cu"])
def test_a_cluster_barrier_precedes_the_first_exchange(source):
    found = 0
    for name, body in kernels(os.path.join(CSRC, source)):
        first = min((body.find(e) for e in EXCHANGE if e in body), default=-1)
        if first < 0:
            continue
        found += 1
        assert 0 <= body.find("cluster_sync();") < first, f"{name}: exchange before a cluster barrier"
    assert found
