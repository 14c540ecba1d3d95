"""Rotating rows and appending them to a paged cache on the GPU, against the definition.

Tolerance per entry, of the pair (x1, x2) it comes from: the angle's fraction is rounded to fp32 (2^-25 of half a turn,
pi * 2^-25) and its sine and cosine by a step or two (2^-23): 2^-22 of |x1| + |x2| together; two products and a sum in
fp32: 2^-23 of it; the frequency, a double, is off by 2^-52 of it: position * frequency * 2^-51.  bf16 outputs: 2^-8 of
their magnitude.
"""

import numpy as np
import pytest
import torch

import speculative_decoding_step_gb300 as pe
from oracle import mx, packed

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _np(t):
    return t.detach().double().cpu().numpy()


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _cfg(n_q, n_kv, hd, dtype, theta=1e4, B=1, max_pages=1):
    return pe.Config.make(B, 1, 64, n_q, n_kv, hd, 64, 2, 1, max_pages, dtype, rope_theta=theta)


def _tol(x, positions, axis, theta, dtype, want):
    half = x.shape[-1] // 2
    size = np.abs(x[..., :half]) + np.abs(x[..., half:])
    freq = theta ** (-np.arange(half) / half)
    turn = np.abs(positions[axis].T.astype(np.float64)) * freq * 2.0 ** -51
    one = size * (2.0 ** -22 + 2.0 ** -23 + turn[:, None])
    tol = np.concatenate([one, one], -1)
    return tol + HALF[dtype] * (np.abs(want) + tol)


def _rows(rng, n, n_q, n_kv, hd, dtype):
    """q, k, v side by side in one buffer, as a fused projection leaves them."""
    both = torch.from_numpy(rng.standard_normal((n, (n_q + 2 * n_kv) * hd + 16))).cuda().to(DT[dtype])
    return both, both[:, :n_q * hd], both[:, n_q * hd:(n_q + n_kv) * hd], both[:, (n_q + n_kv) * hd:(n_q + 2 * n_kv) * hd]


CASES = [(1, 1, 1, 64), (3, 8, 2, 64), (17, 5, 1, 128), (64, 64, 8, 64), (130, 32, 4, 128), (40, 3, 3, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("axes,theta", [(1, 1e4), (3, 1e4), (2, 5e5), (1, 0.5)])
@pytest.mark.parametrize("n,n_q,n_kv,hd", CASES)
def test_append_against_the_definition(dtype, axes, theta, n, n_q, n_kv, hd):
    rng = np.random.default_rng(n * 31 + n_q + axes)
    cfg = _cfg(n_q, n_kv, hd, dtype, theta)
    both, q, k, v = _rows(rng, n, n_q, n_kv, hd, dtype)
    src = both.clone()
    positions = rng.integers(0, 200000, (axes, n)).astype(np.int32)
    positions[0, 0] = 0
    axis = rng.integers(0, axes, hd // 2)
    pages = n // 16 + 3
    slots = rng.permutation(pages * 16)[:n].astype(np.int64)
    slots[n // 2::5] = -1
    kc = torch.from_numpy(rng.standard_normal((pages, 16, n_kv, hd))).cuda().to(DT[dtype])
    vc = torch.from_numpy(rng.standard_normal((pages, 16, n_kv, hd))).cuda().to(DT[dtype])
    kb, vb = _np(kc).reshape(-1, n_kv, hd), _np(vc).reshape(-1, n_kv, hd)
    out, err = torch.full((n, n_q * hd), 7.0, device="cuda", dtype=DT[dtype]), _err()
    pos = torch.from_numpy(positions if axes > 1 else positions[0]).cuda()
    pe.append_kv(cfg, q, k, v, pos, torch.from_numpy(slots).cuda(), (kc, vc), out, err,
                 axes=bytes(axis.tolist()) if axes > 1 else None)
    assert int(err.item()) == 0 and torch.equal(both, src)
    if axes == 1:
        axis[:] = 0
    qn, kn = _np(q).reshape(n, n_q, hd), _np(k).reshape(n, n_kv, hd)
    want = mx.rotated(qn, positions, axis, theta)
    assert (np.abs(_np(out).reshape(n, n_q, hd) - want) <= _tol(qn, positions, axis, theta, dtype, want)).all()
    want = mx.rotated(kn, positions, axis, theta)
    tol = _tol(kn, positions, axis, theta, dtype, want)
    keep = slots >= 0
    kg, vg = _np(kc).reshape(-1, n_kv, hd), _np(vc).reshape(-1, n_kv, hd)
    assert (np.abs(kg[slots[keep]] - want[keep]) <= tol[keep]).all()
    assert np.array_equal(vg[slots[keep]], _np(v).reshape(n, n_kv, hd)[keep])
    rest = np.ones(pages * 16, bool)
    rest[slots[keep]] = False
    assert np.array_equal(kg[rest], kb[rest]) and np.array_equal(vg[rest], vb[rest])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_largest_number_of_heads_and_axes(dtype):
    rng = np.random.default_rng(4)
    n, n_q, n_kv, hd = 3, 4096, 512, 128
    cfg = _cfg(n_q, n_kv, hd, dtype)
    _, q, k, v = _rows(rng, n, n_q, n_kv, hd, dtype)
    positions, axis = rng.integers(0, 5000, (8, n)).astype(np.int32), rng.integers(0, 8, hd // 2)
    kc, vc = (torch.zeros((1, 16, n_kv, hd), device="cuda", dtype=DT[dtype]) for _ in range(2))
    out, err = torch.empty((n, n_q * hd), device="cuda", dtype=DT[dtype]), _err()
    pe.append_kv(cfg, q, k, v, torch.from_numpy(positions).cuda(), torch.arange(n, device="cuda"), (kc, vc), out, err,
                 axes=bytes(axis.tolist()))
    assert int(err.item()) == 0 and torch.equal(vc[0, :n].flatten(1), v)
    for got, x, h in ((out, q, n_q), (kc[0, :n], k, n_kv)):
        xn = _np(x).reshape(n, h, hd)
        want = mx.rotated(xn, positions, axis, 1e4)
        assert (np.abs(_np(got).reshape(n, h, hd) - want) <= _tol(xn, positions, axis, 1e4, dtype, want)).all()


@pytest.mark.parametrize("hd", [64, 128])
def test_far_and_negative_positions(hd):
    rng = np.random.default_rng(hd)
    positions = np.array([[0, 1, -1, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31, 123456789]], np.int32)
    n = positions.shape[1]
    cfg = _cfg(2, 1, hd, "f32")
    _, q, k, v = _rows(rng, n, 2, 1, hd, "f32")
    kc, vc = (torch.zeros((1, 16, 1, hd), device="cuda") for _ in range(2))
    out, err = torch.empty((n, 2 * hd), device="cuda"), _err()
    pe.append_kv(cfg, q, k, v, torch.from_numpy(positions[0]).cuda(), torch.arange(n, device="cuda"), (kc, vc), out, err)
    axis = np.zeros(hd // 2, int)
    for got, x, h in ((out, q, 2), (kc[0, :n], k, 1)):
        xn = _np(x).reshape(n, h, hd)
        want = mx.rotated(xn, positions, axis, 1e4)
        assert (np.abs(_np(got).reshape(n, h, hd) - want) <= _tol(xn, positions, axis, 1e4, "f32", want)).all()
    assert np.array_equal(_np(out[0]), _np(q[0]))  # position 0 turns nothing


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_without_queries_and_bad_slots(dtype):
    rng = np.random.default_rng(2)
    cfg = _cfg(4, 2, 64, dtype)
    n = 20
    both, q, k, v = _rows(rng, n, 4, 2, 64, dtype)
    pos = torch.arange(n, device="cuda", dtype=torch.int32) * 1000
    slots = torch.arange(n, device="cuda")
    slots[3], slots[4], slots[5] = 32, -2, 1 << 40
    caches = [[torch.full((2, 16, 2, 64), 5.0, device="cuda", dtype=DT[dtype]) for _ in range(2)] for _ in range(3)]
    out, err = torch.empty((n, 256), device="cuda", dtype=DT[dtype]), _err()
    pe.append_kv(cfg, q, k, v, pos, slots, caches[0], out, err)
    assert int(err.item()) == pe.PE_DEV_BAD_PAGE
    assert bool((caches[0][0].view(-1, 128)[3:6] == 5).all()) and bool((caches[0][1].view(-1, 128)[3:6] == 5).all())
    pe.append_kv(cfg, None, k, v, pos, slots, caches[1], None, err)
    pe.append_kv(cfg, q, k, v, pos, slots, caches[2], q, err)  # queries over themselves
    assert torch.equal(q, out)
    for c in caches[1:]:
        assert torch.equal(c[0], caches[0][0]) and torch.equal(c[1], caches[0][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,n_q,n_kv,hd", [(1, 2, 1, 64), (37, 64, 8, 64), (130, 12, 3, 128), (300, 5, 5, 64), (4100, 20, 20, 128),
                                          (9000, 40, 40, 64)])
def test_packed_append_is_append_then_pack(dtype, n, n_q, n_kv, hd):
    rng = np.random.default_rng(n + hd)
    cfg = _cfg(n_q, n_kv, hd, dtype)
    _, q, k, v = _rows(rng, n, n_q, n_kv, hd, dtype)
    pages = n // 16 + 2
    slots = torch.from_numpy(rng.permutation(pages * 16)[:n].astype(np.int64)).cuda()
    slots[n // 2::3] = -1
    pos = torch.from_numpy(rng.integers(0, 100000, (2, n)).astype(np.int32)).cuda()
    axes = bytes(rng.integers(0, 2, hd // 2).tolist())
    err = _err()
    out = [torch.empty((n, n_q * hd), device="cuda", dtype=DT[dtype]) for _ in range(2)]
    pool = [torch.full((pages, n_kv, 18 * hd), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pe.append_kv(cfg, q, k, v, pos, slots, pool[0], out[0], err, axes=axes)
    # the same rows rotated into a plain cache, one slot each, then packed from there
    room = [torch.empty((n // 16 + 1, 16, n_kv, hd), device="cuda", dtype=DT[dtype]) for _ in range(2)]
    pe.append_kv(cfg, q, k, v, pos, torch.arange(n, device="cuda"), room, out[1], err, axes=axes)
    rows = [c.view(-1, n_kv * hd)[:n] for c in room]
    pe.pack_kv(cfg, rows[0], rows[1], slots, pool[1], err)
    assert torch.equal(out[0], out[1]) and torch.equal(pool[0], pool[1]) and int(err.item()) == 0


def test_caches_beyond_4_gib():
    """Slots whose bytes lie beyond 32 bits."""
    pages, n_kv, hd = 150000, 8, 128  # 150000 * 16 * 8 * 128 * 2 bytes = 4.9 GB each
    cfg = _cfg(8, n_kv, hd, "bf16")
    kc, vc = (torch.zeros((pages, 16, n_kv, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _, q, k, v = _rows(np.random.default_rng(1), 3, 8, n_kv, hd, "bf16")
    slots = torch.tensor([pages * 16 - 1, 5, pages * 16 - 17], device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, err = torch.empty((3, 8 * hd), dtype=torch.bfloat16, device="cuda"), _err()
    pe.append_kv(cfg, q, k, v, pos, slots, (kc, vc), out, err)
    assert torch.equal(kc.view(-1, n_kv * hd)[slots], k) and torch.equal(vc.view(-1, n_kv * hd)[slots], v)
    assert torch.equal(out, q) and int(err.item()) == 0 and int(torch.count_nonzero(kc.view(-1, n_kv * hd).any(1))) == 3


def test_captured_append_replays_with_new_rows():
    rng = np.random.default_rng(3)
    cfg = _cfg(8, 2, 64, "bf16")
    n = 33
    both, q, k, v = _rows(rng, n, 8, 2, 64, "bf16")
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    slots = torch.arange(n, device="cuda")
    cache = [torch.zeros((4, 16, 2, 64), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    other = [torch.zeros_like(c) for c in cache]
    out, want, err = torch.empty((n, 512), device="cuda", dtype=torch.bfloat16), None, _err()
    want = torch.empty_like(out)
    pe.append_kv(cfg, q, k, v, pos, slots, cache, out, err)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pe.append_kv(cfg, q, k, v, pos, slots, cache, out, err)
    for i in range(3):
        both.copy_(torch.randn_like(both))
        pos += 100
        g.replay()
        pe.append_kv(cfg, q, k, v, pos, slots, other, want, err)
        assert torch.equal(out, want) and torch.equal(cache[0], other[0]) and torch.equal(cache[1], other[1])
    assert int(err.item()) == 0


def test_a_layer_of_calls():
    """Projection in 4 bits, rotation into a packed cache, attention, projection back with the residual: each call's
    output is what the next one takes, and each is checked against its definition on what it took."""
    rng = np.random.default_rng(11)
    B, n_q, n_kv, hd, d = 3, 8, 2, 64, 320
    lens, rows = [5, 40, 17], [5, 9, 1]
    n = sum(rows)
    cfg = _cfg(n_q, n_kv, hd, "bf16", B=B, max_pages=4)
    err = _err()
    wqkv = 0.05 * rng.standard_normal(((n_q + 2 * n_kv) * hd, d)).astype(np.float32)
    wo = 0.05 * rng.standard_normal((d, n_q * hd)).astype(np.float32)
    mats = []
    for w in (wqkv, wo):
        m = pe.MxMatrix(*w.shape)
        pe.quantize_mx(torch.from_numpy(w).cuda(), m, err)
        mats.append(m)
    ws = pe.alloc_linear_mx_workspace(n, max(d, n_q * hd))
    table = torch.from_numpy(rng.permutation(12).reshape(3, 4).astype(np.int32)).cuda()
    pool = pe.alloc_packed_pool(cfg, 12)
    old = [L - r for L, r in zip(lens, rows)]
    # what is cached already
    for b in range(B):
        if old[b]:
            p = torch.arange(old[b], device="cuda")
            kv = torch.from_numpy(rng.standard_normal((2, old[b], n_kv * hd))).cuda().bfloat16()
            pe.pack_kv(cfg, kv[0], kv[1], table[b][p // 16].long() * 16 + p % 16, pool, err)
    x = torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).cuda().bfloat16()
    resid = torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).cuda()
    seq = torch.from_numpy(np.repeat(np.arange(B), rows)).cuda()
    pos = torch.cat([torch.arange(o, L) for o, L in zip(old, lens)]).int().cuda()
    slots = table[seq, (pos // 16).long()].long() * 16 + pos % 16
    start = torch.tensor(np.cumsum([0] + rows), dtype=torch.int32, device="cuda")
    qkv = torch.empty((n, (n_q + 2 * n_kv) * hd), device="cuda", dtype=torch.bfloat16)
    q = torch.empty((n, n_q * hd), device="cuda", dtype=torch.bfloat16)
    att = torch.empty_like(q)
    y = resid.clone()

    pe.linear_mx(x, mats[0], qkv, ws, err)
    cut = [qkv[:, :n_q * hd], qkv[:, n_q * hd:(n_q + n_kv) * hd], qkv[:, (n_q + n_kv) * hd:]]
    pe.append_kv(cfg, *cut, pos, slots, pool, q, err)
    pe.attend_packed(cfg, q, pool, table, start, pos, max(rows), att, pe.alloc_attend_workspace(cfg), err)
    pe.linear_mx(att, mats[1], y, ws, err, add=y)
    assert int(err.item()) == 0

    xk, wk = mx.kept(_np(x)), mx.kept(wqkv)
    want, size = xk @ wk.T, np.abs(xk) @ np.abs(wk).T
    assert (np.abs(_np(qkv) - want) <= d * 2.0 ** -23 * size + 2.0 ** -8 * (np.abs(want) + d * 2.0 ** -23 * size)).all()
    qn = _np(cut[0]).reshape(n, n_q, hd)
    positions, axis = pos.cpu().numpy()[None], np.zeros(hd // 2, int)
    want = mx.rotated(qn, positions, axis, 1e4)
    assert (np.abs(_np(q).reshape(n, n_q, hd) - want) <= _tol(qn, positions, axis, 1e4, "bf16", want)).all()
    kk, vv = packed.read(pool.cpu().numpy(), slots.cpu().numpy())
    assert np.array_equal(vv.reshape(n, -1), packed.kept(_np(cut[2]).reshape(n, n_kv, hd)).reshape(n, -1))
    # attention over what the pool keeps: weights rounded to bf16, output too (2^-8 each), fp32 in between
    for i in range(n):
        b, L = int(seq[i]), int(pos[i]) + 1
        p = np.arange(L)
        at = table[b].cpu().numpy()[p // 16] * 16 + p % 16
        kb, vb = packed.read(pool.cpu().numpy(), at)
        for h in range(n_q):
            s = kb[:, h // 4] @ _np(q)[i, h * hd:(h + 1) * hd] / 8
            wgt = np.exp(s - s.max())
            wgt /= wgt.sum()
            want, size = wgt @ vb[:, h // 4], wgt @ np.abs(vb[:, h // 4])
            got = _np(att)[i, h * hd:(h + 1) * hd]
            assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2 * 2.0 ** -8 + 2.0 ** -12) * size).all()
    ak, wk = mx.kept(_np(att)), mx.kept(wo)
    want, size = ak @ wk.T + _np(resid), np.abs(ak) @ np.abs(wk).T + np.abs(_np(resid))
    assert (np.abs(_np(y) - want) <= (n_q * hd + 1) * 2.0 ** -23 * size + 2.0 ** -24 * np.abs(want)).all()


def test_python_refusals():
    cfg = _cfg(2, 1, 64, "bf16")
    _, q, k, v = _rows(np.random.default_rng(0), 4, 2, 1, 64, "bf16")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    slots, err = torch.arange(4, device="cuda"), _err()
    cache = [torch.zeros((1, 16, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out = torch.empty((4, 128), dtype=torch.bfloat16, device="cuda")
    bad = [dict(axes=b"\0" * 31), dict(axes=[0] * 32), dict(positions=pos.long()), dict(positions=pos[:3]),
           dict(slots=slots.int()), dict(q_out=None), dict(cache=(cache[0], cache[1].float())),
           dict(cache=torch.zeros((1, 1, 17 * 64), dtype=torch.uint8, device="cuda")), dict(k=k.float()),
           dict(q=q[:3])]
    good = dict(q=q, k=k, v=v, positions=pos, slots=slots, cache=cache, q_out=out, err=err)
    pe.append_kv(cfg, **good)
    for change in bad:
        with pytest.raises((ValueError, AttributeError)):
            pe.append_kv(cfg, **{**good, **change})
    with pytest.raises(pe.PeError):
        pe.append_kv(cfg, **{**good, "axes": b"\1" * 32})
