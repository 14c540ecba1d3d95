"""Drafter rounds with the LM head in 4 bits on the GPU.

The rows that reach the LM head are read out of a pass whose LM head is the identity (each logit is then one product by
one, so exact), and the logits of the pass with the 4-bit head are held to the definition in 64 bits on those rows, with
the products' tolerance: d * 2^-23 * sum |x w| (that many fp32 additions, each off by at most a step, of exact terms).
"""

import numpy as np
import pytest
import torch

import speculative_decoding_step_gb300 as pe
from oracle import mx
from pe_workload import Config

from gpu_harness import run_stages, setup
from test_gpu_packed_drafter import _packed

pytestmark = pytest.mark.gpu


def _cfg(**kw) -> Config:
    base = dict(name="mx-head", B=3, K=4, n_layers=1, d=256, n_q=8, n_kv=2, head_dim=64, ffn=384, vocab=1000,
                dtype="bf16", prefix="uniform", prefix_args=(1, 300), accepted="uniform", seed=81)
    base.update(kw)
    return Config(**base)


CASES = {
    "few-rows": _cfg(),
    "one-row": _cfg(B=1, K=1, vocab=300, seed=82),
    "kept-rows-odd-vocabulary": _cfg(B=9, K=7, d=320, vocab=5003, seed=83),      # 63 rows, kept as they are in 4 bits
    "kept-rows-f32": _cfg(B=2, K=7, d=264, vocab=777, dtype="f32", seed=84),     # a width that ends inside a block
    "stages": _cfg(B=12, K=8, vocab=2000, seed=85),                               # 96 rows
    "wide": _cfg(B=40, K=8, d=256, vocab=20000, prefix_args=(1, 40), seed=86),    # 320 rows, tiles of 256
    "wide-f32": _cfg(B=40, K=8, d=260, vocab=20000, dtype="f32", prefix_args=(1, 40), seed=87),
    "two-layers-hd128": _cfg(B=2, K=8, n_q=16, n_kv=2, head_dim=128, d=512, n_layers=2, seed=88),
}


def _matrix(t):
    m = pe.MxMatrix(*t.shape)
    m.data.fill_(255)  # rows beyond the vocabulary: scales that are no numbers
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pe.quantize_mx(t, m, err)
    assert int(err.item()) == 0
    return m


def _with_head(c, head):
    c.weights = pe.DeviceWeights(**{**c.W, "lm_head": head})
    c.rd = pe.Round(c.cfg, c.weights, c.kv, c.Rd["block_table"])


def _start(c, packed):
    if packed:
        c.kv = _packed(c)
    buffers = c.kv.pools if packed else c.kv.k_cache + c.kv.v_cache
    return buffers, [b.clone() for b in buffers]


@pytest.mark.parametrize("packed", [False, True], ids=["plain", "packed"])
@pytest.mark.parametrize("name", list(CASES))
def test_logits_and_drafts_of_the_4_bit_head(name, packed):
    c = setup(CASES[name])
    buffers, start = _start(c, packed)
    T, V, d = c.cfg.B * c.cfg.K, c.cfg.vocab, c.cfg.d
    assert V >= d
    eye = torch.zeros_like(c.W["lm_head"])
    eye[:d].fill_diagonal_(1)
    _with_head(c, eye)
    assert run_stages(c) == 0
    rows = c.rd.logits[:, :d].cpu().numpy()
    after = [b.clone() for b in buffers]
    for b, s in zip(buffers, start):
        b.copy_(s)
    _with_head(c, _matrix(c.W["lm_head"]))
    c.rd.workspace.fill_(0xA5)
    assert run_stages(c) == 0
    assert all(torch.equal(a, b) for a, b in zip(after, buffers))  # the cache does not depend on the LM head
    x, w = mx.kept(rows), mx.kept(c.W["lm_head"].float().cpu().numpy())
    got, want, size = c.rd.logits.double().cpu().numpy(), x @ w.T, np.abs(x) @ np.abs(w).T
    assert np.all(np.abs(got - want) <= d * 2.0 ** -23 * size)
    assert np.array_equal(c.rd.draft_tokens.cpu().numpy().reshape(-1), got.argmax(1))
    drafts = c.rd.draft_tokens.clone()
    c.rd.draft_tokens.fill_(-1)
    assert run_stages(c, logits=False) == 0 and torch.equal(drafts, c.rd.draft_tokens)


def test_equal_logits_go_to_the_lowest_token():
    c = setup(_cfg(B=40, K=8, vocab=3000, prefix_args=(1, 40), seed=89))
    head = c.W["lm_head"].clone()
    head[1000:2000] = head[:1000]
    head[2000:] = head[:1000]
    _with_head(c, _matrix(head))
    assert run_stages(c) == 0
    assert int(c.rd.draft_tokens.max()) < 1000
    _with_head(c, _matrix(torch.zeros_like(head)))
    assert run_stages(c) == 0
    assert int(c.rd.draft_tokens.abs().max()) == 0


@pytest.mark.parametrize("packed", [False, True], ids=["plain", "packed"])
@pytest.mark.parametrize("name", ["few-rows", "kept-rows-f32", "kept-rows-odd-vocabulary", "wide"])
def test_step_equals_the_stages_and_its_captured_graph(name, packed):
    c = setup(CASES[name])
    buffers, start = _start(c, packed)
    _with_head(c, _matrix(c.W["lm_head"]))
    R = c.Rd
    assert run_stages(c) == 0
    targets = torch.cat([c.rd.draft_tokens, torch.full((c.cfg.B, 1), 3, dtype=torch.int32, device="cuda")], 1)
    targets[0, 0] += 1
    targets %= c.cfg.vocab
    c.rd.verify(targets)
    want = [t.clone() for t in [c.rd.draft_tokens, c.rd.logits, c.rd.out["num_accepted"], c.rd.out["bonus"]] + buffers]

    def same():
        assert int(c.rd.err.item()) == 0
        have = [c.rd.draft_tokens, c.rd.logits, c.rd.out["num_accepted"], c.rd.out["bonus"]] + buffers
        assert all(torch.equal(a, b) for a, b in zip(have, want))

    def reset():
        for b, s in zip(buffers, start):
            b.copy_(s)
        c.rd.draft_tokens.fill_(-1)
        c.rd.logits.zero_()
        c.rd.workspace.fill_(0xA5)

    def step():
        c.rd.step(R["prev_tokens"], R["prev_pos"], R["num_accepted"], R["bonus"], R["target_hidden"], targets, logits=True)

    reset()
    step()
    same()
    reset()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        reset()
        g.replay()
        same()


def test_logits_that_are_no_numbers_are_reported():
    c = setup(CASES["few-rows"])
    m = _matrix(c.W["lm_head"])
    m.data[mx.scale_at(5, 0)] = 255
    _with_head(c, m)
    assert run_stages(c) == pe.PE_DEV_NONFINITE


def test_heads_and_workspaces_that_are_refused():
    c = setup(CASES["few-rows"])
    m = _matrix(c.W["lm_head"])
    _with_head(c, m)
    with pytest.raises(pe.PeError):  # the plain calls' workspace is too short
        pe.draft_forward(c.cfg, c.weights, c.kv, c.Rd["block_table"], c.rd.x0, c.rd.meta, pe.alloc_workspace(c.cfg),
                         c.rd.draft_tokens, c.rd.err)
    with pytest.raises(pe.PeError):
        pe.draft_forward_noalloc(c.cfg, c.weights, c.kv, c.Rd["block_table"], c.rd.x0, c.rd.meta, c.rd.draft_tokens,
                                 c.rd.err)
    _with_head(c, m.first(999))
    with pytest.raises(ValueError):
        c.rd.forward()
