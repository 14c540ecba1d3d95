"""What the kernels' sources have to keep to for their launches to overlap safely.

A kernel may start while the one before it still runs (programmatic dependent launch), once every CTA of that one has
triggered it or ended.  The tensor-core kernels allocate tensor memory before they wait for the kernel before them, and an
allocation waits, without a limit, until the SM has room: a kernel that triggered its successor before its own allocation
could wait for tensor memory that the successor holds while it waits for this kernel.
"""

import glob
import os
import re

import pytest

import speculative_decoding_step_gb300 as pe

CSRC = os.path.join(os.path.dirname(pe.__file__), "csrc")


def _kernels():
    """(file, name, body) of every kernel, without comments."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for part in re.split(r"^__global__", text, flags=re.M)[1:]:
            body = part.split("\n}\n")[0]
            yield os.path.basename(path), re.search(r"(\w+)\s*\(\s*const ", body).group(1), body


ALLOCATING = [k for k in _kernels() if re.search(r"\btmem_alloc\w*\(", k[2])]


def test_the_tensor_core_kernels_are_found():
    assert {name for _, name, _ in ALLOCATING} >= {"gemm_tc_kernel", "attn_bf16_kernel", "attend_tile_kernel"}


@pytest.mark.parametrize("file,name,body", ALLOCATING, ids=[f"{f}:{n}" for f, n, _ in ALLOCATING])
def test_tensor_memory_is_allocated_before_the_next_kernel_may_start(file, name, body):
    alloc = [m.start() for m in re.finditer(r"\btmem_alloc\w*\(", body)]
    trigger = [m.start() for m in re.finditer(r"\bpdl_trigger\(\)", body)]
    assert trigger, "an untriggered kernel needs no such order, but all of these trigger"
    assert max(alloc) < min(trigger)
    # one thread's trigger counts for its CTA, so a barrier of the CTA stands between the two
    assert "__syncthreads();" in body[max(alloc):min(trigger)]
