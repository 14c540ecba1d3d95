"""The packed KV cache without a GPU: the format's definition, and what the calls refuse before
anything is launched (placeholder pointers, never dereferenced: every call here stops at a check
or has no rows)."""

import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_step_gb300 as pe
from oracle import packed


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("values", [False, True])
def test_rows_hold_every_entry_once(hd, values):
    assert sorted(packed.nibble_of(hd, values)) == list(range(hd))


def test_kept_values_are_within_half_a_scale_and_exact_in_bf16():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 128)) * np.exp(3 * rng.standard_normal((200, 1)))
    n, byte = packed.quantise(x)
    s = np.repeat(packed.SCALES[byte], 16, axis=-1)
    y = n * s
    inside = np.repeat(np.abs(x).reshape(200, 8, 16).max(-1) <= 7 * packed.SCALES[255], 16, axis=-1)
    assert inside.mean() > 0.9 and np.all(np.abs(x - y)[inside] <= (s / 2)[inside])
    assert np.all(np.abs(y)[~inside] <= 7 * packed.SCALES[255])
    assert np.array_equal(torch.from_numpy(y).bfloat16().double().numpy(), y)
    amax = np.abs(x).reshape(200, 8, 16).max(-1)
    fits = amax <= 7 * packed.SCALES[255]
    assert np.all((7 * packed.SCALES[byte] >= amax)[fits]) and np.all(7 * packed.SCALES[byte - 1] < amax)


def _cfg(**kw):
    base = dict(B=3, K=1, d=64, n_q=8, n_kv=2, head_dim=64, ffn=64, vocab=2, n_layers=1, max_pages_per_seq=9,
                dtype="bf16")
    base.update(kw)
    return pe.Config.make(**base)


def _p(x=1 << 40):
    return ctypes.c_void_p(x)


NULL = ctypes.c_void_p(None)


def _pack(cfg, k=None, v=None, ks=128, vs=128, slots=None, n=0, pool=None, pages=4, err=None):
    d = lambda x: _p() if x is None else x  # noqa: E731
    return pe.lib().pe_pack_kv(ctypes.byref(cfg), d(k), d(v), ks, vs, d(slots), n, d(pool), pages, d(err), NULL)


def _unpack(cfg, k=None, v=None, ks=128, vs=128, slots=None, n=0, pool=None, pages=4, err=None):
    d = lambda x: _p() if x is None else x  # noqa: E731
    return pe.lib().pe_unpack_kv(ctypes.byref(cfg), d(pool), pages, d(slots), n, d(k), d(v), ks, vs, d(err), NULL)


@pytest.mark.parametrize("call", [_pack, _unpack])
def test_pack_and_unpack_refuse_before_launch(call):
    c = _cfg()
    assert call(c) == 0                                   # no rows: fine, and nothing is launched
    for name in ("k", "v", "slots", "pool", "err"):
        assert call(c, **{name: NULL}) == 1
    for name in ("k", "v", "pool"):
        assert call(c, **{name: _p((1 << 40) + 8)}) == 1  # not 16-byte aligned
    for name in ("ks", "vs"):
        assert call(c, **{name: 127}) == 1                # shorter than a row
        assert call(c, **{name: 132}) == 1                # rows not 16-byte aligned
    assert call(c, ks=136, vs=128) == 0
    assert call(c, n=-1) == 2 and call(c, pages=0) == 2
    for bad, status in ((dict(head_dim=96), 3), (dict(page_size=32), 3), (dict(n_q=7), 2), (dict(B=0), 2),
                        (dict(n_kv=0), 2), (dict(max_pages_per_seq=0), 2)):
        assert call(_cfg(**bad)) == status, bad
    assert pe.lib().pe_pack_kv(None, _p(), _p(), 128, 128, _p(), 0, _p(), 4, _p(), NULL) == 1


def test_unpack_refuses_outputs_that_overlap():
    c, at = _cfg(), 1 << 40
    assert _unpack(c, k=_p(at), v=_p(at), n=3) == 1
    assert _unpack(c, k=_p(at), v=_p(at + 2 * 128 * 2), n=3) == 1          # the third row of the other
    assert _unpack(c, k=_p(at), v=_p(at + 240), ks=256, vs=256, n=3) == 1  # side by side, 16 bytes short
    assert _unpack(c, k=_p(at), v=_p(at + 256), ks=256, vs=264, n=3) == 1


def _attend(cfg, q=None, qs=512, pool=None, pages=4, table=None, start=None, pos=None, n=0, most=1, out=None, os=512,
            ws=None, ws_bytes=0, err=None):
    d = lambda x, at: _p((1 << 40) + at * (1 << 32)) if x is None else x  # noqa: E731
    return pe.lib().pe_attend_packed(ctypes.byref(cfg), d(q, 0), qs, d(pool, 1), pages, d(table, 2), d(start, 3),
                                     d(pos, 4), n, most, d(out, 5), os, d(ws, 6), ctypes.c_size_t(ws_bytes), d(err, 7),
                                     NULL)


def test_attend_refuses_before_launch():
    c = _cfg()
    full = pe.attend_workspace_bytes(c)
    assert full > 0 and pe.packed_page_bytes(c) == 2 * 18 * 64
    assert _attend(c, ws_bytes=full) == 0                 # no rows
    assert _attend(c, ws_bytes=full - 1) == 2
    for name in ("q", "pool", "table", "start", "pos", "out", "ws", "err"):
        assert _attend(c, ws_bytes=full, **{name: NULL}) == 1
    for name in ("q", "pool", "out"):
        assert _attend(c, ws_bytes=full, **{name: _p((1 << 40) + 4)}) == 1
    assert _attend(c, ws_bytes=full, ws=_p((1 << 40) + 128)) == 1
    assert _attend(c, ws_bytes=full, qs=504) == 1 and _attend(c, ws_bytes=full, os=516) == 1
    assert _attend(c, ws_bytes=full, n=-1) == 2 and _attend(c, ws_bytes=full, pages=0) == 2
    assert _attend(c, ws_bytes=full, n=65537) == 2
    assert _attend(c, ws_bytes=full, n=4, most=0) == 2
    # output rows over the query rows, whole or in part; a short workspace stops the calls that may pass
    q = (1 << 40)
    assert _attend(c, ws_bytes=full, n=4, most=4, q=_p(q), out=_p(q)) == 1
    assert _attend(c, ws_bytes=full, n=4, most=4, q=_p(q), out=_p(q + 3 * 1024)) == 1
    assert _attend(c, ws_bytes=full, n=4, most=4, q=_p(q), qs=1024, out=_p(q + 1008), os=1024) == 1
    assert pe.attend_workspace_bytes(_cfg(head_dim=96)) == 0 and pe.packed_page_bytes(_cfg(B=0)) == 0
    # bounds that B * max_rows rows make far too many tiles of
    assert _attend(_cfg(B=60000), ws_bytes=full, n=65536, most=65536) == 2
    # the sizes that only the drafter reads do not matter here
    assert _attend(_cfg(d=7, ffn=1, K=1, vocab=2, n_layers=1), ws_bytes=full) == 0


def test_python_calls_refuse_what_is_not_on_the_gpu():
    c = _cfg()
    pool = torch.zeros((4, 2, 18 * 64), dtype=torch.uint8)
    x, slots, err = torch.zeros(5, 2, 64).bfloat16(), torch.zeros(5, dtype=torch.int64), torch.zeros(1).int()
    if torch.cuda.is_available():
        pytest.skip("the same checks run on the GPU")
    with pytest.raises((ValueError, RuntimeError)):
        pe.pack_kv(c, x, x, slots, pool, err)
    with pytest.raises((ValueError, RuntimeError)):
        pe.unpack_kv(c, pool, slots, x, x, err)
