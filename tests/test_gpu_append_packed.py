"""Appending rotated rows to a packed pool: against the definition, with slots outside the pool and entries that are no
numbers.

A rotated key is off by the tolerance that test_gpu_append.py derives, t.  The pool keeps it as one of the codes -7..7 of its
block's scale s: what is kept of the exact rotation, computed in 64 bits, and what the pool holds differ where t moves a key
across the middle between two codes (a step of s) or its block's largest across the border of a scale (the scales' bytes then
differ by one, and each kept value is half a step off its own key).  So the value read back is within s/2 + t of the exact
key, s being the scale that the pool holds (its codes then reach 7 s, which is at least the block's largest less t), and the
scale is that of an amax within t of the exact one.
"""

import numpy as np
import pytest
import torch

import speculative_decoding_step_gb300 as pe
from oracle import mx, packed
from test_gpu_append import DT, _cfg, _err, _np, _rows, _tol

pytestmark = pytest.mark.gpu


def _close_keys(got, byte, want, tol):
    """Read-back keys [n][heads][hd] and their scale bytes [n][heads][hd/16] against exact rotated keys and t."""
    blocks = want.shape[:-1] + (want.shape[-1] // packed.BLOCK, packed.BLOCK)
    w, t = want.reshape(blocks), tol.reshape(blocks)
    finite = np.isfinite(w)
    size = np.where(finite, np.abs(w), 0)
    slack = np.where(finite, t, 0).max(-1)
    low = np.searchsorted(7 * packed.SCALES, np.maximum(size.max(-1) - slack, 0), side="left")
    high = np.searchsorted(7 * packed.SCALES, size.max(-1) + slack, side="left")
    assert ((low <= byte) & (byte <= np.minimum(high, 255))).all()
    s = packed.SCALES[byte][..., None]
    g = got.reshape(blocks)
    # what is no number is kept as 0, what is infinite as the block's largest code
    exact = np.where(np.isnan(w), 0, np.where(np.isinf(w), np.sign(w) * 7 * s, np.where(finite, w, 0)))
    room = np.where(finite, s / 2 + t, 0)
    assert (np.abs(g - exact) <= room).all(), np.argwhere(~(np.abs(g - exact) <= room))[:5]


def _scales(pool, slots, hd):
    return pool[..., 16 * hd:17 * hd].reshape(*pool.shape[:2], packed.PAGE, hd // 16)[slots // 16, :, slots % 16]


CASES = [(1, 2, 1, 64), (2, 2, 1, 128), (37, 8, 8, 64), (130, 12, 3, 128), (300, 5, 5, 64), (2100, 20, 20, 128), (9000, 4, 4, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("queries", [False, True])
@pytest.mark.parametrize("n,n_q,n_kv,hd", CASES)
def test_packed_append_against_the_definition(dtype, queries, n, n_q, n_kv, hd):
    rng = np.random.default_rng(n + hd + 7)
    cfg = _cfg(n_q, n_kv, hd, dtype)
    _, q, k, v = _rows(rng, n, n_q, n_kv, hd, dtype)
    pages = n // 16 + 2
    slots = rng.permutation(pages * 16)[:n].astype(np.int64)
    slots[n // 3::7] = -1
    positions, axis = rng.integers(0, 100000, (2, n)).astype(np.int32), rng.integers(0, 2, hd // 2)
    before = rng.integers(0, 256, (pages, n_kv, 18 * hd), dtype=np.uint8)
    pool, err = torch.from_numpy(before).cuda(), _err()
    out = torch.full((n, n_q * hd), float("nan"), device="cuda", dtype=DT[dtype]) if queries else None
    pe.append_kv(cfg, q if queries else None, k, v, torch.from_numpy(positions).cuda(), torch.from_numpy(slots).cuda(), pool,
                 out, err, axes=bytes(axis.tolist()))
    assert int(err.item()) == 0
    after, keep = pool.cpu().numpy(), slots >= 0
    if keep.any():
        kn, vn = _np(k).reshape(n, n_kv, hd)[keep], _np(v).reshape(n, n_kv, hd)[keep]
        pos = positions[:, keep]
        want = mx.rotated(kn, pos, axis, 1e4)
        got = packed.read(after, slots[keep])
        _close_keys(got[0], _scales(after, slots[keep], hd), want, _tol(kn, pos, axis, 1e4, dtype, want))
        assert np.array_equal(got[1], packed.kept(vn))
    rest = ~packed.entry_bytes(after.shape, slots[keep])
    assert np.array_equal(after[rest], before[rest])
    if queries:
        qn = _np(q).reshape(n, n_q, hd)
        want = mx.rotated(qn, positions, axis, 1e4)
        assert (np.abs(_np(out).reshape(n, n_q, hd) - want) <= _tol(qn, positions, axis, 1e4, dtype, want)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,n_kv,hd", [(40, 2, 64), (40, 3, 128), (9000, 4, 128)])
def test_slots_outside_the_pool_are_reported_and_passed_over(dtype, n, n_kv, hd):
    rng = np.random.default_rng(n + hd)
    cfg = _cfg(n_kv, n_kv, hd, dtype)
    _, _, k, v = _rows(rng, n, n_kv, n_kv, hd, dtype)
    pages = n // 16 + 1
    good = torch.arange(n, device="cuda")
    bad = {3: pages * 16, 4: -2, 5: 1 << 40, n - 1: -(1 << 40), 17: (1 << 63) - 1, 18: -(1 << 63)}
    pos = torch.arange(n, device="cuda", dtype=torch.int32) * 3
    first = torch.randint(0, 256, (pages, n_kv, 18 * hd), device="cuda", dtype=torch.uint8)
    pools, err = [first.clone() for _ in range(3)], _err()
    pe.append_kv(cfg, None, k, v, pos, good, pools[0], None, err)
    passed = good.clone()
    passed[list(bad)] = -1
    pe.append_kv(cfg, None, k, v, pos, passed, pools[1], None, err)
    assert int(err.item()) == 0
    out_of_it = good.clone()
    for row, slot in bad.items():
        out_of_it[row] = slot
    pe.append_kv(cfg, None, k, v, pos, out_of_it, pools[2], None, err)
    assert int(err.item()) == pe.PE_DEV_BAD_PAGE and torch.equal(pools[1], pools[2])
    mask = packed.entry_bytes(first.shape, np.array(list(bad)))
    assert np.array_equal(pools[2].cpu().numpy()[mask], first.cpu().numpy()[mask])
    assert np.array_equal(pools[2].cpu().numpy()[~mask], pools[0].cpu().numpy()[~mask])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
def test_entries_that_are_no_numbers_are_reported_and_kept_as_such(dtype, hd):
    rng = np.random.default_rng(hd)
    n, n_kv = 24, 3
    cfg = _cfg(n_kv, n_kv, hd, dtype)
    _, _, k, v = _rows(rng, n, n_kv, n_kv, hd, dtype)
    nan, inf = float("nan"), float("inf")
    k[2, 5], k[3, hd + 40], k[4, 2 * hd + 7], k[7, hd - 1], k[8, 0] = nan, inf, -inf, -inf, nan
    k[9, :hd] = nan
    k[10, hd:2 * hd] = inf
    v[1, 3], v[5, hd + 9], v[6, 33] = nan, inf, -inf
    v[11, :16] = nan
    pos = torch.arange(1, n + 1, device="cuda", dtype=torch.int32) * 11
    slots, err = torch.arange(n, device="cuda"), _err()
    pool = torch.zeros((2, n_kv, 18 * hd), device="cuda", dtype=torch.uint8)
    pe.append_kv(cfg, None, k, v, pos, slots, pool, None, err)
    assert int(err.item()) == pe.PE_DEV_NONFINITE
    kn, vn = _np(k).reshape(n, n_kv, hd), _np(v).reshape(n, n_kv, hd)
    axis, p = np.zeros(hd // 2, int), pos.cpu().numpy()[None]
    with np.errstate(invalid="ignore"):
        want = mx.rotated(kn, p, axis, 1e4)
        tol = np.nan_to_num(_tol(np.nan_to_num(kn, posinf=0, neginf=0), p, axis, 1e4, dtype, np.nan_to_num(want, posinf=0,
                                                                                                          neginf=0)))
        values = packed.quantise(vn)
    after = pool.cpu().numpy()
    got = packed.read(after, np.arange(n))
    _close_keys(got[0], _scales(after, np.arange(n), hd), want, tol)
    assert np.array_equal(got[1], values[0] * np.repeat(packed.SCALES[values[1]], 16, axis=-1))
