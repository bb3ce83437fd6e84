"""Programmatic dependent launch and tensor memory, by reading the sources: a
block lets the next kernel of its stream launch only once it holds its own
columns.  (The other way round a dependent on the same SM can allocate first and
wait for this grid, which waits for the columns.)"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_kv_cache_append_b200", "csrc")


def kernels(path):
    """(name, body) of every __global__ function, comments taken out."""
    src = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"__global__\s+void\s+([^;{]*?)(\w+)\s*\(", src):
        i = src.index("{", m.end())
        depth, j = 0, i
        while True:
            depth += {"{": 1, "}": -1}.get(src[j], 0)
            j += 1
            if depth == 0:
                break
        name = re.sub(r"__launch_bounds__\s*\(.*?\)\s*(?=\w+$)", "", m.group(2))
        yield name, src[i:j]


TMEM = [(os.path.basename(f), k, body) for f in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) for k, body in kernels(f)
        if "tmem_alloc(" in body]


def test_the_kernels_are_found():
    assert len(TMEM) >= 7


@pytest.mark.parametrize("file,name,body", TMEM, ids=[f"{f}-{i}" for i, (f, _, _) in enumerate(TMEM)])
def test_dependents_launch_behind_the_allocation(file, name, body):
    triggers = [m.start() for m in re.finditer(r"pdl_launch_dependents\(\)", body)]
    assert triggers and min(triggers) > body.index("tmem_alloc("), file
    first = body[body.index("tmem_alloc("):min(triggers)]
    # the allocating warp itself, or everyone behind a barrier
    assert "}" not in first or "__syncthreads()" in first, file
