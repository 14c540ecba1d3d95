"""Pipeline waits that run out in the 4-bit products whose CTAs share a tile, and in the drafter's 4-bit LM head.

As in test_gpu_failure.py the host shortens the wait limit and has one launch leave a pipeline stage of its first CTA unarmed.
That CTA gives up and still has to reach the barriers at which its cluster exchanges partial sums; the head's last CTA still
turns what there is into drafts.  The call returns, PE_DEV_TIMEOUT is set, and the same call passes afterwards.
"""

import time

import numpy as np
import pytest
import torch

import speculative_decoding_step_gb300 as pe
from gpu_harness import run_stages, setup
from test_gpu_mx_head import CASES, _cfg, _matrix, _with_head

pytestmark = pytest.mark.gpu


class _Short:
    """The next launch of a tensor-core product lacks a stage, and waits give up after a millisecond."""

    def __init__(self, stage):
        self.stage = stage

    def __enter__(self):
        pe.set_wait_limit_ns(1_000_000)
        pe.skip_pipeline_stage_for_test(self.stage)
        self.start = time.perf_counter()

    def __exit__(self, *_):
        torch.cuda.synchronize()
        pe.skip_pipeline_stage_for_test(-1)
        pe.set_wait_limit_ns(0)
        assert time.perf_counter() - self.start < 1.0


# rows, features, width: x kept as records or rounded in the product; x in the stages; eight, four and two CTAs a tile
SHARED = {
    "eight-kept": (16, 128, 8192), "eight-rounded": (8, 128, 4096), "eight-stages": (128, 500, 8192),
    "many-tiles-stages": (128, 2000, 8192), "four-kept": (9, 3000, 5000), "two-kept": (7, 7000, 5000),
}


@pytest.mark.parametrize("stage", [0, 1])
@pytest.mark.parametrize("name", list(SHARED))
@pytest.mark.parametrize("add", [False, True])
def test_a_shared_tile_whose_first_cta_gives_up(name, stage, add):
    n, m, w = SHARED[name]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(n + m)
    x = torch.randn(n, w, device="cuda", generator=g)
    wm = pe.MxMatrix(m, w)
    pe.quantize_mx(torch.randn(m, w, device="cuda", generator=g), wm, err)
    ws = pe.alloc_linear_mx_workspace(n, w)
    a = torch.randn(n, m, device="cuda", generator=g) if add else None
    want, y = torch.empty((n, m), device="cuda"), torch.empty((n, m), device="cuda")
    pe.linear_mx(x, wm, want, ws, err, add=a)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and not bool(want.isnan().any())
    one_stage = name == "eight-rounded"  # four pieces of the width a CTA: its only stage
    with _Short(0 if one_stage else stage):
        pe.linear_mx(x, wm, y, ws, err, add=a)
    assert int(err.item()) == pe.PE_DEV_TIMEOUT
    err.zero_()
    for _ in range(2):
        y.fill_(float("nan"))
        pe.linear_mx(x, wm, y, ws, err, add=a)
        assert int(err.item()) == 0 and torch.equal(y, want)


# The products of an fp32 drafter's layers are not on the tensor cores, so the head's is the launch that gives up.  Stages are
# counted from the CTA's first on; wide-f32's first CTA fills four, one a tile.
HEADS = {"kept": CASES["kept-rows-f32"], "stages": CASES["wide-f32"],
         "pairs": _cfg(B=56, K=8, d=2560, vocab=20000, dtype="f32", prefix_args=(1, 40), seed=90)}


@pytest.mark.parametrize("name,stage", [("kept", 0), ("stages", 0), ("stages", 1), ("stages", 3), ("pairs", 0), ("pairs", 7)])
def test_a_4_bit_head_that_gives_up(name, stage):
    c = setup(HEADS[name])
    R, K = c.Rd, c.cfg.K
    _with_head(c, _matrix(c.W["lm_head"]))
    assert run_stages(c) == 0
    drafts, logits = c.rd.draft_tokens.clone(), c.rd.logits.clone()
    targets = torch.cat([drafts, torch.full((c.cfg.B, 1), 3, dtype=torch.int32, device="cuda")], 1)

    def reset():
        for now, before in zip(c.kv.k_cache + c.kv.v_cache, c.k_before + c.v_before):
            now.copy_(before)
        c.rd.err.zero_()
        c.rd.draft_tokens.fill_(-7)

    def step():
        c.rd.step(R["prev_tokens"], R["prev_pos"], R["num_accepted"], R["bonus"], R["target_hidden"], targets, logits=True)
        torch.cuda.synchronize()

    for call in (lambda: run_stages(c), step):
        reset()
        with _Short(stage):
            call()
        assert int(c.rd.err.item()) == pe.PE_DEV_TIMEOUT
        reset()
        call()
        assert int(c.rd.err.item()) == 0
        assert torch.equal(c.rd.draft_tokens, drafts) and torch.equal(c.rd.logits, logits)
    assert np.array_equal(c.rd.out["num_accepted"].cpu().numpy(), np.full(c.cfg.B, K))
