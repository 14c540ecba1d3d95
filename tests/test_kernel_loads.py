"""How kernels may read what an earlier call wrote.

A kernel may start while the one before it still writes (programmatic dependent launch), and waits for it before it reads.
Loads through the read-only path (__ldg, ld.global.nc, or __restrict__ parameters that the compiler turns into them) are
for data that nobody writes while the kernel runs, its wait included: a 32-byte sector that the SM's cache took in for the
earlier kernel, which half of it belonged to, need not be looked up again.  The operators on rows that a caller may have
written with the call before use none.  (No GPU: the sources are read.)"""

import glob
import os
import re

import pytest

import speculative_decoding_step_gb300 as pe

CSRC = os.path.join(os.path.dirname(pe.__file__), "csrc")
FILES = sorted(f for kind in ("pe_mx", "pe_append", "pe_packed") for f in glob.glob(os.path.join(CSRC, kind + "*.cu*")))


def test_the_files_are_found():
    assert {os.path.basename(f) for f in FILES} >= {"pe_mx.cu", "pe_mx.cuh", "pe_mx_gemm.cu", "pe_mx_gemm.cuh",
                                                    "pe_mx_pair.cu", "pe_append.cu", "pe_packed.cu", "pe_packed_attn.cu"}


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(f) for f in FILES])
def test_no_loads_through_the_read_only_path(path):
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ldg\b|\.nc\.|\.nc\b|__restrict__", text)
