"""Tensor memory and dependent launch, read from the sources: a kernel that
allocates tensor memory lets the next kernel start only after its allocation
(the allocation waits without a limit for columns that the next kernel's CTAs,
waiting for this one, may hold)."""
import glob
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "driven_collective_communication_gb300", "csrc")


def code(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


def kernels():
    """(file, body from its launch bounds to the next kernel) of all that allocate."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        for body in re.split(r"\b__global__\b", code(path))[1:]:
            if "tcgen05.alloc" in body:
                found.append(pytest.param(body, id=os.path.basename(path)))
    return found


def test_every_allocating_kernel_is_looked_at():
    files = [p for p in glob.glob(os.path.join(CSRC, "*.cu*")) if "tcgen05.alloc" in code(p)]
    assert len(files) >= 4 and len(kernels()) == len(files)


@pytest.mark.parametrize("body", kernels())
def test_the_next_kernel_starts_after_the_allocation(body):
    assert "pdl_prologue" not in body and "launch_dependents" not in body
    alloc = body.index("tcgen05.alloc")
    trigger = [m.start() for m in re.finditer(r"\bpdl_trigger\(\)", body)]
    assert len(trigger) == 1 and body.count("tcgen05.alloc") == 1
    between = body[alloc:trigger[0]]
    assert "__syncthreads();" in between  # every thread triggers after warp-wide allocation
    assert "pdl_wait();" in body[:trigger[0]]
