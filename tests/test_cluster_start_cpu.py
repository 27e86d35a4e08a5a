"""Distributed shared memory: a block of a cluster may touch another one's shared
memory only when that block runs.  Being scheduled together does not mean that each
has begun, so every kernel that reaches into its peers waits at a cluster barrier
before its first access.  Read from the sources: nothing here touches a device."""
import glob
import os
import re

import pytest

from routed_grouped_gemm_routing_gb300 import build

CSRC = build.CSRC
REMOTE = re.compile(r"(?:st|ld|red|atom)(?:\.\w+)*\.shared::cluster\.(?!global)|\bload_peer\(")
WAIT = re.compile(r"barrier\.cluster\.wait|\bcluster_sync\(\)")


def _kernels(text):
    """(name, body) of every __global__ function."""
    for m in re.finditer(r"__global__ void", text):
        name = re.search(r"(\w+)\s*\((?=[^()]*(?:\([^()]*\)[^()]*)*\)\s*\{)", text[m.end():])
        at = text.index("{", m.end() + name.end())
        depth, i = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
            if depth == 0:
                break
        yield name.group(1), text[at:i]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu*")))


def test_the_kernels_are_found():
    names = {n for f in _sources() for n, _ in _kernels(open(f).read())}
    assert {"decode_router_kernel", "few_rows_kernel", "rn_bwd_kernel", "linear_dz_kernel"} <= names


@pytest.mark.parametrize("path", _sources(), ids=os.path.basename)
def test_a_barrier_before_the_first_access_to_a_peer(path):
    for name, body in _kernels(open(path).read()):
        code = re.sub(r"//[^\n]*", "", body)
        first = REMOTE.search(code)
        if first:
            wait = WAIT.search(code)
            assert wait and wait.start() < first.start(), f"{name} reaches into its peers before it knows that they run"
