"""Clusters of CTAs that hold tensor memory while they wait for one another.

Such a CTA has all of its SM's tensor memory from its start to its end, and an allocation waits without a limit.  If two of
them fitted an SM, two calls on two streams could each have a CTA that waits for tensor memory which the other's holds while
that one waits for its cluster.  So each asks for more than half of an SM's shared memory (asked of the library's own plan;
no GPU)."""

import ctypes
import os
import re

import speculative_decoding_step_gb300 as pe

SM, OWN = 228 * 1024, 1024  # an SM's shared memory, and what every CTA takes of it besides
CSRC = os.path.join(os.path.dirname(pe.__file__), "csrc")


def _smem(n_rows, n_out, width, sms=152):
    f = getattr(pe.lib(), "_ZN2pe14mx_matmul_smemEiiiiPi")
    f.restype, cluster = ctypes.c_size_t, ctypes.c_int()
    return int(f(n_rows, n_out, width, sms, ctypes.byref(cluster))), cluster.value


def test_ctas_that_share_a_tile_of_a_product_have_an_sm_each():
    seen = set()
    for n in (1, 7, 16, 17, 33, 64, 65, 100, 128, 129, 200, 300):
        for m in (1, 128, 300, 768, 2000, 5000, 20000):
            for w in [128 * k for k in (1, 2, 5, 8, 11, 16, 23, 32, 40, 47, 64, 100, 300, 1000)] + [1 << 20]:
                smem, cluster = _smem(n, m, w)
                if cluster > 1:
                    seen.add((cluster, n <= 64))
                    assert 2 * (smem + OWN) > SM, (n, m, w, cluster, smem)
                assert smem + OWN <= SM
    assert seen == {(c, k) for c in (2, 4, 8) for k in (False, True)}  # every size of cluster, x kept or in the stages


def test_pairs_of_ctas_have_an_sm_each():
    """The pair kernel's shared memory is a constant of its source: stages of 8 records' worth fill the SM."""
    text = open(os.path.join(CSRC, "pe_mx_pair.cu")).read()
    assert re.search(r"kPairStages = \(kTcSmemOptIn - 128 - \(int\)kMxgCtrl\) / \(int\)kPairStage;", text)
    record, scales, ctrl, opt_in = 8704, 512, 1024 + 2048, 232448
    stage = 2 * record + 2 * (record - scales) + 2 * 2 * scales
    smem = 128 + (opt_in - 128 - ctrl) // stage * stage + ctrl
    assert 2 * (smem + OWN) > SM and smem <= opt_in
