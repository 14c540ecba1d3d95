"""The drafter round over a packed KV cache on the GPU, against the 64-bit oracle.

The oracle's pass takes every key and value from the caches as the GPU's pass left them, so that its logits depend
continuously on what the GPU computed (an entry next to a rounding boundary may land on either side of it), and the
logits are held to the drafter's own tolerance.  The entries that the pass wrote are held to the oracle's k and v: at most
half a scale away from what the storage tolerance allows, with the smallest scale that fits.
"""

import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_step_gb300 as pe
from oracle import packed
from pe_workload import Config, f32_to_bf16, make_round
from pe_workload.device import to_torch

from gpu_harness import KV_TOL, check_logits, meta_np, run_stages, setup

pytestmark = pytest.mark.gpu


def _cfg(**kw) -> Config:
    base = dict(name="packed", B=3, K=4, n_layers=1, d=256, n_q=8, n_kv=2, head_dim=64, ffn=384, vocab=1000,
                dtype="bf16", prefix="uniform", prefix_args=(1, 300), accepted="uniform", seed=61)
    base.update(kw)
    return Config(**base)


CASES = {
    "bf16-hd64": _cfg(),                                                              # tiles of the tensor cores
    "bf16-hd64-L2-few-rows": _cfg(B=5, K=1, n_layers=2, seed=62),                     # at most 8 query vectors
    "bf16-hd64-16-vectors": _cfg(B=2, K=2, seed=63),
    "bf16-hd128-L2": _cfg(B=2, K=8, n_q=16, n_kv=2, head_dim=128, d=512, n_layers=2, seed=64),
    "bf16-one-head-each": _cfg(B=4, K=5, n_q=3, n_kv=3, seed=65),
    "bf16-short": _cfg(B=6, K=3, prefix_args=(1, 2), seed=66),
    "bf16-many-rows": _cfg(B=24, K=8, d=320, ffn=448, prefix_args=(1, 60), seed=67),  # GEMMs on CTA pairs
    "f32-hd64-L2": _cfg(dtype="f32", n_layers=2, seed=68),
    "f32-hd128": _cfg(dtype="f32", head_dim=128, B=2, seed=69),
}


def _packed(c):
    """The case's caches packed by pack_kv, as a DevicePackedKV."""
    pages = c.kv.k_cache[0].shape[0]
    slots = torch.arange(pages * 16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pools = []
    for k, v in zip(c.kv.k_cache, c.kv.v_cache):
        pool = pe.alloc_packed_pool(c.cfg, pages)
        pe.pack_kv(c.cfg, k.reshape(pages * 16, -1), v.reshape(pages * 16, -1), slots, pool, err)
        pools.append(pool)
    assert int(err.item()) == 0
    return pe.DevicePackedKV(pools)


def _setup(cfg_np, rnd=None):
    c = setup(cfg_np, rnd=rnd)
    c.kv = _packed(c)
    c.rd = pe.Round(c.cfg, c.weights, c.kv, c.Rd["block_table"])
    return c, [p.cpu().numpy() for p in c.kv.pools]


def _check_entries(cfg, pool, before, slots, want_k, want_v):
    """The entries at slots against what was to be packed, and every other byte as before."""
    stray = (pool != before) & ~packed.entry_bytes(pool.shape, slots)
    assert not stray.any()
    tol = KV_TOL[cfg.dtype]
    for got, want, base in zip(packed.read(pool, slots), (want_k, want_v), (16 * cfg.head_dim, 17 * cfg.head_dim)):
        nb = cfg.head_dim // 16
        page, off = np.asarray(slots) // 16, np.asarray(slots) % 16
        byte = pool[..., base:base + cfg.head_dim].reshape(*pool.shape[:2], 16, nb)[page, :, off]
        scale = packed.SCALES[byte]
        store = tol * np.maximum(1, np.abs(want))
        assert np.all(np.abs(got - want) <= np.repeat(scale / 2, 16, axis=-1) + store)
        amax = (np.abs(want) + store).reshape(*want.shape[:-1], nb, 16).max(-1)
        assert np.all((scale <= 9 / 8 * amax / 7) | (byte == 0))


def _draft_rows(cfg, num_accepted, rows):
    at, S = {int(r): i for i, r in enumerate(rows)}, 2 * cfg.K
    return [at[r] for b in range(cfg.B)
            for r in [b * S + int(num_accepted[b])] + [b * S + cfg.K + m for m in range(1, cfg.K)]]


@pytest.mark.parametrize("name", list(CASES))
def test_round_over_a_packed_cache_against_oracle(name):
    c, before = _setup(CASES[name])
    cfg, r = c.cfg_np, c.r_np
    assert run_stages(c) == 0
    pools = [p.cpu().numpy() for p in c.kv.pools]
    meta = meta_np(c)
    n = int(meta["n_valid"][0])
    rows = meta["row_list"][:n]
    x0 = oracle.scatter_hidden(c.w_np.emb, c.w_np.h_shared, r.target_hidden, meta["input_ids"], meta["is_mask"],
                               meta["hidden_map"])
    ref = packed.draft_forward(cfg, c.w_np, x0[rows], meta["positions"][rows], rows // (2 * cfg.K), r.block_table, pools,
                               _draft_rows(cfg, r.num_accepted, rows))
    for l in range(cfg.n_layers):
        _check_entries(cfg, pools[l], before[l], meta["slot_mapping"][rows], ref["new_k"][l], ref["new_v"][l])
    ref["drafts"] = oracle.argmax_lowest(ref["logits"]).reshape(cfg.B, cfg.K)
    check_logits(c, ref)


@pytest.mark.parametrize("name", ["bf16-hd64", "bf16-hd64-L2-few-rows", "bf16-hd128-L2", "f32-hd64-L2"])
def test_step_equals_the_stages_and_its_captured_graph(name):
    c, _ = _setup(CASES[name])
    R = c.Rd
    start = [p.clone() for p in c.kv.pools]
    assert run_stages(c, logits=True) == 0
    targets = c.rd.draft_tokens.clone()
    targets = torch.cat([targets, torch.full((c.cfg.B, 1), 3, dtype=torch.int32, device="cuda")], 1)
    targets[0, 0] += 1
    targets %= c.cfg.vocab
    c.rd.verify(targets)
    want = dict(drafts=c.rd.draft_tokens.clone(), logits=c.rd.logits.clone(), pools=[p.clone() for p in c.kv.pools],
                acc=c.rd.out["num_accepted"].clone(), bonus=c.rd.out["bonus"].clone())

    def same():
        assert int(c.rd.err.item()) == 0
        assert torch.equal(c.rd.draft_tokens, want["drafts"]) and torch.equal(c.rd.logits, want["logits"])
        assert torch.equal(c.rd.out["num_accepted"], want["acc"]) and torch.equal(c.rd.out["bonus"], want["bonus"])
        assert all(torch.equal(a, b) for a, b in zip(c.kv.pools, want["pools"]))

    def reset():
        for p, q in zip(c.kv.pools, start):
            p.copy_(q)
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


def test_loop_of_rounds_in_place_and_replayed():
    """Three rounds whose state overwrites itself, as calls and as replays of one graph."""
    cfg_np = _cfg(B=4, K=3, n_layers=2, prefix_args=(20, 90), seed=70)
    rnd = make_round(cfg_np)
    c, _ = _setup(cfg_np, rnd)
    R = c.Rd
    start = [p.clone() for p in c.kv.pools]
    state0 = {k: R[k].clone() for k in ("prev_tokens", "prev_pos", "num_accepted", "bonus")}
    hidden, targets = torch.empty_like(R["target_hidden"]), torch.empty((4, 4), dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    feeds = [(torch.randn(hidden.shape, generator=g).to(hidden.dtype).cuda(),
              torch.randint(0, cfg_np.vocab, (4, 4), generator=g, dtype=torch.int32).cuda()) for _ in range(3)]

    def run(one):
        for p, q in zip(c.kv.pools, start):
            p.copy_(q)
        for k in state:
            state[k].copy_(state0[k])
        seen = []
        for h, t in feeds:
            hidden.copy_(h)
            targets.copy_(t)
            one()
            seen.append([c.rd.draft_tokens.clone()] + [state[k].clone() for k in sorted(state)])
        return seen + [[p.clone() for p in c.kv.pools]]

    state = {k: v.clone() for k, v in state0.items()}
    calls = run(lambda: c.rd.step_inplace(state, hidden, targets))
    graph = c.rd.capture_loop(state, hidden, targets)
    replays = run(graph.replay)
    assert int(c.rd.err.item()) == 0
    for a, b in zip(calls, replays):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert bool((calls[0][3] != calls[2][3]).any())


@pytest.mark.parametrize("name", ["bf16-hd64", "bf16-hd128-L2", "f32-hd64-L2", "bf16-many-rows"])
def test_inject_kv_into_a_packed_cache(name):
    cfg = CASES[name]
    rnd = make_round(cfg)
    rnd.num_accepted[0] = 0
    c, before = _setup(cfg, rnd)
    w32 = (np.random.default_rng(7).standard_normal((cfg.d, cfg.d)) * 0.02).astype(np.float32)
    w_inj = f32_to_bf16(w32) if cfg.dtype == "bf16" else w32
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    R = c.Rd
    pe.inject_kv(c.cfg, c.weights, to_torch(w_inj), c.kv, R["block_table"], R["prev_pos"], R["num_accepted"],
                 R["target_hidden"], c.rd.workspace, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    ref = oracle.inject_kv(cfg, c.w_np, w_inj, rnd.target_hidden, rnd.prev_pos, rnd.num_accepted, rnd.block_table)
    shape = (len(ref["slots"]), cfg.n_kv, cfg.head_dim)
    for l in range(cfg.n_layers):
        _check_entries(cfg, c.kv.pools[l].cpu().numpy(), before[l], ref["slots"], ref["new_k"][l].reshape(shape),
                       ref["new_v"][l].reshape(shape))


def test_bad_page_is_reported_and_the_other_sequences_keep_their_drafts():
    cfg = _cfg(B=3, prefix_args=(60, 120), seed=71)
    rnd = make_round(cfg)
    c, _ = _setup(cfg, rnd)
    assert run_stages(c) == 0
    want = c.rd.draft_tokens.clone()
    c2, _ = _setup(cfg, rnd)
    c2.rd.block_table = c2.Rd["block_table"].clone()
    c2.rd.block_table[1, 0] = c2.kv.pools[0].shape[0]  # past the pool, in the prefix
    assert run_stages(c2) == pe.PE_DEV_BAD_PAGE
    assert torch.equal(c2.rd.draft_tokens[[0, 2]], want[[0, 2]])


def test_python_calls_refuse_pools_of_another_config():
    c, _ = _setup(_cfg())
    pages = c.kv.pools[0].shape[0]
    two_layers = pe.Config.make(3, 4, 256, 8, 2, 64, 384, 1000, 2, c.cfg.max_pages_per_seq, "bf16")
    R = c.Rd
    for cfg, kv in ((two_layers, c.kv),
                    (c.cfg, pe.DevicePackedKV([torch.zeros((pages, 1, 18 * 64), dtype=torch.uint8, device="cuda")]))):
        with pytest.raises(ValueError):
            pe.step(cfg, c.weights, kv, R["block_table"], R["prev_tokens"], R["prev_pos"], R["num_accepted"],
                    R["bonus"], R["target_hidden"], R["prev_tokens"], c.rd.workspace, c.rd.out, c.rd.err)
    with pytest.raises(pe.PeError):  # the plain calls' workspace is too short
        pe.draft_forward(c.cfg, c.weights, c.kv, R["block_table"], c.rd.x0, c.rd.meta, pe.alloc_workspace(c.cfg),
                         c.rd.draft_tokens, c.rd.err)
