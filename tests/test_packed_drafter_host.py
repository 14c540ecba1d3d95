"""The drafter over a packed cache without a GPU: the oracle's two passes agree, and what the calls refuse
before anything is launched."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_step_gb300 as pe
from oracle import packed
from pe_workload import Config, make_round, make_weights


def test_oracle_pass_over_a_packed_cache_is_the_drafter_pass_on_what_it_keeps():
    """With a cache of kept values and the pass's own rows kept in it, the packed pass equals the drafter pass whose
    new rows are those kept values (one layer: the rows' k and v do not depend on the cache)."""
    cfg = Config(name="packed-host", B=2, K=3, n_layers=1, d=64, n_q=4, n_kv=2, head_dim=64, ffn=96, vocab=120,
                 dtype="f32", prefix="uniform", prefix_args=(1, 40), accepted="uniform", seed=3)
    w, rnd = make_weights(cfg), make_round(cfg)
    plain = oracle.run_round(cfg, w, rnd, want_kv=True)
    rows, meta = plain["rows"], plain["meta"]
    pages = rnd.k_cache[0].shape[0]
    shape = (-1, cfg.n_kv, cfg.head_dim)
    pool = np.zeros((pages, cfg.n_kv, 18 * cfg.head_dim), dtype=np.uint8)
    every = np.arange(pages * 16)
    packed.write(pool, rnd.k_cache[0].reshape(shape), rnd.v_cache[0].reshape(shape), every)
    slots = meta["slot_mapping"][rows]
    packed.write(pool, plain["new_k"][0].reshape(shape), plain["new_v"][0].reshape(shape), slots)
    seqs = rows // (2 * cfg.K)
    idx = {int(r): i for i, r in enumerate(rows)}
    dr = [idx[int(rows_b)] for b in range(cfg.B)
          for rows_b in [b * 6 + int(rnd.num_accepted[b])] + [b * 6 + 3 + m for m in range(1, 3)]]
    got = packed.draft_forward(cfg, w, plain["x0"][rows], meta["positions"][rows], seqs, rnd.block_table, [pool], dr)
    assert np.allclose(got["new_k"][0].reshape(len(rows), -1), plain["new_k"][0], atol=1e-12)
    assert np.allclose(got["new_v"][0].reshape(len(rows), -1), plain["new_v"][0], atol=1e-12)
    # the same pass, row by row, with oracle.attend over the kept entries
    k, v = packed.read(pool, every)
    X = oracle.linear(oracle.widen(plain["x0"][rows]) if plain["x0"].dtype != np.float64 else plain["x0"][rows], w.fc)
    Y = oracle.rmsnorm(X, w.norm_attn[0], cfg.rms_eps)
    q = oracle.linear(Y, np.ascontiguousarray(w.wqkv[0][:cfg.n_q * 64]))
    out = np.zeros((len(rows), cfg.n_q * 64))
    for i, r in enumerate(rows):
        p = int(meta["positions"][r])
        at = np.arange(p + 1)
        s = rnd.block_table[seqs[i], at // 16].astype(np.int64) * 16 + at % 16
        for h in range(cfg.n_q):
            qh = oracle.rope(q[i, h * 64:(h + 1) * 64], p, cfg.rope_theta)
            out[i, h * 64:(h + 1) * 64] = oracle.attend(qh, k[s, h // 2], v[s, h // 2], 64 ** -0.5)
    X = X + oracle.linear(out, w.wo[0])
    gu = oracle.linear(oracle.rmsnorm(X, w.norm_mlp[0], cfg.rms_eps), w.w_gate_up[0])
    act = np.array([[oracle.silu(g) * u for g, u in zip(a[:cfg.ffn], a[cfg.ffn:])] for a in gu])
    X = X + oracle.linear(act, w.w_down[0])
    want = oracle.linear(oracle.rmsnorm(X[dr], w.norm_final, cfg.rms_eps), w.lm_head)
    assert np.allclose(got["logits"], want, atol=1e-9)


def _cfg(**kw):
    base = dict(B=2, K=3, d=128, n_q=8, n_kv=2, head_dim=64, ffn=128, vocab=300, n_layers=2, max_pages_per_seq=9,
                dtype="bf16")
    base.update(kw)
    return pe.Config.make(**base)


def _p(i):
    return ctypes.c_void_p((1 << 40) + i * (1 << 32))


def _weights(n_layers):
    arrs = [(ctypes.c_void_p * n_layers)(*[(1 << 50) + 4096 * (l + 1) for l in range(n_layers)]) for _ in range(6)]
    p = (1 << 50)
    return pe._Weights(p, p, p, *arrs, p, p), arrs


def _kv(pools, num_pages=40):
    arr = (ctypes.c_void_p * len(pools))(*pools)
    return pe._PackedKV(arr, num_pages), arr


def test_packed_workspace_serves_every_call():
    c = _cfg()
    assert pe.packed_workspace_bytes(c) >= pe.workspace_bytes(c) + pe.attend_workspace_bytes(c)
    assert pe.packed_workspace_bytes(_cfg(head_dim=96)) == 0
    assert pe.packed_workspace_bytes(_cfg(d=100)) == 0             # no drafter of this width
    assert pe.packed_workspace_bytes(_cfg(max_pages_per_seq=(1 << 24) + 1)) == 0


@pytest.mark.parametrize("name", ["pe_draft_forward_packed", "pe_step_packed", "pe_inject_kv_packed"])
def test_packed_drafter_calls_refuse_before_launch(name):
    c = _cfg()
    w, keep_w = _weights(2)
    need = pe.packed_workspace_bytes(c)
    n_ptr = {"pe_draft_forward_packed": 7, "pe_step_packed": 7, "pe_inject_kv_packed": 4}[name]
    n_out = {"pe_draft_forward_packed": 3, "pe_step_packed": 7, "pe_inject_kv_packed": 1}[name]

    def call(cfg=c, kv=None, ws=None, ws_bytes=need, drop=None):
        kv = _kv([1 << 49, 1 << 49])[0] if kv is None else kv
        ptrs = [_p(i) for i in range(n_ptr)]
        outs = [_p(20 + i) for i in range(n_out)]
        if drop is not None:
            ptrs[drop] = None
        head = [ctypes.byref(cfg), ctypes.byref(w)]
        head += [_p(30)] if name == "pe_inject_kv_packed" else []
        return getattr(pe.lib(), name)(*head, ctypes.byref(kv), *ptrs, _p(40) if ws is None else ws,
                                       ctypes.c_size_t(ws_bytes), *outs, None)

    assert call(ws_bytes=need - 1) == 2
    assert call(ws_bytes=pe.workspace_bytes(c)) == 2               # the plain calls' workspace is too short
    assert call(ws=ctypes.c_void_p((1 << 40) + 128)) == 1
    for i in range(n_ptr):
        assert call(drop=i) == 1
    for pools, pages in (([1 << 49, 0], 40), ([1 << 49, (1 << 49) + 8], 40), ([1 << 49, 1 << 49], 0)):
        kv, keep = _kv(pools, pages)
        assert call(kv=kv) == 1, (pools, pages)
    assert call(kv=pe._PackedKV(None, 40)) == 1
    assert call(cfg=_cfg(page_size=32)) == 3
    assert call(cfg=_cfg(max_pages_per_seq=(1 << 24) + 1)) == 2    # the packed calls' bound
    del keep_w


def test_device_packed_kv_takes_gpu_pools_only():
    with pytest.raises(ValueError):
        pe.DevicePackedKV([torch.zeros((4, 2, 18 * 64), dtype=torch.uint8)])
    with pytest.raises(ValueError):
        pe.DevicePackedKV([])
