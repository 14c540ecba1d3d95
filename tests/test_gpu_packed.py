"""The packed (4-bit) KV cache on the GPU: pack_kv, unpack_kv and attend_packed against the format's
definition in 64 bits.

Packing is compared byte for byte and reading back value for value.  The attention's tolerance
is derived per element from what it may round (u = 2^-24, half a step of fp32):
  scores     a sum of head_dim products in fp32, times the scale, and the exponent's own error:
             the weight is off by at most 2 * (hd + 8) * u * depth + 2^-20 relative, depth the largest
             sum of |q_e k_e| / sqrt(hd) over the row's positions (bf16 keys and queries are exact);
  sums       over the row's L positions: L * u of the sum of magnitudes, twice (weights, products);
  bf16       each weight is rounded to bf16: 2^-8 of it, and the output: 2^-8 of its magnitude.
All but the last act on `size`, the same weighted sum over the values' magnitudes; the output is
a ratio, so what acts on the weights counts twice.
"""

import numpy as np
import pytest
import torch

import speculative_decoding_step_gb300 as pe
from oracle import packed

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _cfg(B, n_q, n_kv, hd, dtype, max_pages):
    return pe.Config.make(B, 1, 64, n_q, n_kv, hd, 64, 2, 1, max_pages, dtype)


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _dt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _np(t):
    return t.detach().double().cpu().numpy()


# ----------------------------------------------------------------------------- packing and reading back

def _rows(rng, n, n_kv, hd):
    """Rows with blocks of zeros, of one value, of halves of a scale, of tiny and of huge entries."""
    x = rng.standard_normal((n, n_kv, hd)) * np.exp(2 * rng.standard_normal((n, n_kv, 1)))
    b = x.reshape(n, n_kv, hd // 16, 16)
    kind = rng.integers(0, 8, size=b.shape[:3])
    b[kind == 0] = 0
    b[kind == 1] = np.arange(16) / 2.0 - 3.5 + 0.0 * b[kind == 1]  # 7 s = 4: every half of s
    b[kind == 2] *= 1e-7
    b[kind == 3] *= 4e4
    b[kind == 4] = 7 * packed.SCALES[100] * np.sign(b[kind == 4])
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_kv,hd,n", [(1, 64, 1), (8, 64, 37), (3, 64, 130), (1, 128, 5), (4, 128, 67)])
def test_pack_and_unpack_match_the_definition(dtype, n_kv, hd, n):
    rng = np.random.default_rng(n_kv * 1000 + hd + n)
    pages = n // 16 + 3
    cfg = _cfg(1, n_kv, n_kv, hd, dtype, pages)
    slots = rng.permutation(pages * 16)[:n].astype(np.int64)
    slots[n // 2::5] = -1
    ks = n_kv * hd * 2 + 16  # keys and values side by side, as a fused projection leaves them
    both = torch.zeros((n, ks), device="cuda", dtype=_dt(dtype))
    both[:, :n_kv * hd] = torch.from_numpy(_rows(rng, n, n_kv, hd)).reshape(n, -1).cuda()
    both[:, n_kv * hd:2 * n_kv * hd] = torch.from_numpy(_rows(rng, n, n_kv, hd)).reshape(n, -1).cuda()
    k, v = both[:, :n_kv * hd], both[:, n_kv * hd:2 * n_kv * hd]
    before = torch.from_numpy(rng.integers(0, 256, (pages, n_kv, 18 * hd), dtype=np.uint8))
    pool, err = before.cuda(), _err()
    s = torch.from_numpy(slots).cuda()
    pe.pack_kv(cfg, k, v, s, pool, err)
    want = before.numpy().copy()
    packed.write(want, _np(k).reshape(n, n_kv, hd), _np(v).reshape(n, n_kv, hd), slots)
    assert int(err.item()) == 0
    assert np.array_equal(pool.cpu().numpy(), want)
    # read back what was there before as well, some slots twice, into rows with gaps between them
    again = np.concatenate([slots, rng.integers(0, pages * 16, 9), slots[:1]])
    m = len(again)
    room = torch.full((m, 2, n_kv * hd + 8), 7.0, device="cuda", dtype=_dt(dtype))
    ko, vo = room[:, 0, :n_kv * hd], room[:, 1, :n_kv * hd]
    pe.unpack_kv(cfg, pool, torch.from_numpy(again).cuda(), ko, vo, err)
    wk, wv = packed.read(want, np.maximum(again, 0))
    for got, w in ((ko, wk), (vo, wv)):
        w = np.where((again >= 0)[:, None], w.reshape(m, -1), 7.0)
        assert np.array_equal(_np(got), w)
    assert bool((room[:, :, n_kv * hd:] == 7).all()) and int(err.item()) == 0


def test_pack_rounds_halves_and_neighbours_of_halves_away_from_zero():
    """fp32 entries one step either side of every half of a scale, for every mantissa of the scale."""
    rows = []
    for m in range(8):
        for e in (-9, 0, 5):
            s = (1 + m / 8) * 2.0 ** e
            top = np.float32(7 * s)
            for i in range(7):
                h = np.float32((i + 0.5) * s)
                near = [h, np.nextafter(h, np.float32(0)), np.nextafter(h, np.float32(1e9)), np.float32(i * s)]
                block = [top] + near + [-x for x in near] + [top] * 7
                rows.append(block)
    x = np.array(rows, dtype=np.float32)
    x = np.concatenate([x, np.zeros((-len(x) % 4, 16), np.float32)]).reshape(-1, 1, 64)
    n = len(x)
    cfg = _cfg(1, 1, 1, 64, "f32", n // 16 + 1)
    pool, err = pe.alloc_packed_pool(cfg, n // 16 + 1), _err()
    t = torch.from_numpy(x).cuda()
    pe.pack_kv(cfg, t, -t, torch.arange(n, device="cuda"), pool, err)
    want = np.zeros(tuple(pool.shape), dtype=np.uint8)
    packed.write(want, x.astype(np.float64), -x.astype(np.float64), np.arange(n))
    assert np.array_equal(pool.cpu().numpy(), want) and int(err.item()) == 0


def test_pack_rounds_bf16_halves_away_from_zero():
    """Every half of every scale that is one in bf16, (2i + 1)/2 * s: four bits times four."""
    c = np.arange(8, 256)
    s = packed.SCALES[c]
    halves = np.concatenate([np.arange(7) + 0.5, -(np.arange(7) + 0.5), [7.0, -7.0]])
    x = (s[:, None] * halves).reshape(-1, 1, 16)
    x = np.concatenate([x, np.zeros((-len(x) % 4, 1, 16))]).reshape(-1, 1, 64)
    t = torch.from_numpy(x).cuda().bfloat16()
    assert np.array_equal(_np(t), x)  # none is rounded
    n = len(x)
    cfg = _cfg(1, 1, 1, 64, "bf16", n // 16 + 1)
    pool, err = pe.alloc_packed_pool(cfg, n // 16 + 1), _err()
    pe.pack_kv(cfg, t, -t, torch.arange(n, device="cuda"), pool, err)
    want = np.zeros(tuple(pool.shape), dtype=np.uint8)
    packed.write(want, x, -x, np.arange(n))
    assert np.array_equal(pool.cpu().numpy(), want) and int(err.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pack_device_checks(dtype):
    cfg = _cfg(1, 2, 2, 64, dtype, 4)
    x = torch.randn(6, 2, 64, device="cuda").to(_dt(dtype))
    slots = torch.tensor([0, 64, 5, -2, 17, -1], device="cuda")
    pool, err = torch.full((4, 2, 18 * 64), 255, dtype=torch.uint8, device="cuda"), _err()
    want = pool.cpu().numpy()
    pe.pack_kv(cfg, x, x, slots, pool, err)
    packed.write(want, _np(x), _np(x), np.array([0, -1, 5, -1, 17, -1]))
    assert int(err.item()) == pe.PE_DEV_BAD_PAGE
    assert np.array_equal(pool.cpu().numpy(), want)
    err.zero_()
    out = torch.full((6, 2, 64), 3.0, device="cuda", dtype=_dt(dtype))
    out2 = out.clone()
    pe.unpack_kv(cfg, pool, slots, out, out2, err)
    assert int(err.item()) == pe.PE_DEV_BAD_PAGE
    wk, _ = packed.read(want, np.array([0, 0, 5, 0, 17, 0]))
    keep = np.array([0, 2, 4])
    assert np.array_equal(_np(out)[keep], wk[keep])
    assert bool((out[[1, 3, 5]] == 3).all()) and bool((out2[[1, 3, 5]] == 3).all())
    # NaN and infinities: flagged, kept as 0 and as the block's largest codes
    err.zero_()
    x[2, 1, 3], x[2, 1, 4], x[2, 1, 5] = float("nan"), float("inf"), -float("inf")
    pe.pack_kv(cfg, x, x, torch.arange(6, device="cuda"), pool, err)
    packed.write(want, _np(x), _np(x), np.arange(6))
    assert int(err.item()) == pe.PE_DEV_NONFINITE
    assert np.array_equal(pool.cpu().numpy(), want)


# ----------------------------------------------------------------------------- attention

class Att:
    """A packed cache of random bytes or rows, and ragged query rows over it."""

    def __init__(self, dtype, hd, n_q, n_kv, rows, ctx, seed=0, raw=False, spare=1, empty=(), gap=0, tail=0):
        rng = np.random.default_rng(seed)
        self.n_q, self.n_kv, self.hd, self.dtype = n_q, n_kv, hd, dtype
        B = len(rows)
        pages = [max(1, -(-c // 16)) for c in ctx]
        num = sum(pages) + 2
        perm = rng.permutation(num)
        self.table = np.full((B, max(pages) + spare), -7, dtype=np.int32)
        at = 0
        for b in range(B):
            self.table[b, :pages[b]] = perm[at:at + pages[b]]
            at += pages[b]
        self.start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32) + gap
        n = int(self.start[-1]) + tail
        self.pos = np.full(n, -1, dtype=np.int32)
        for b in range(B):
            z = slice(self.start[b], self.start[b + 1])
            self.pos[z] = np.arange(ctx[b] - rows[b], ctx[b])
        for r in empty:
            self.pos[r] = -1
        if raw:
            # any bytes are a cache; scales around 2^-3 keep the scores in range
            self.pool = rng.integers(0, 256, (num, n_kv, 18 * hd), dtype=np.uint8)
            self.pool[..., 16 * hd:] = rng.integers(110, 140, (num, n_kv, 2 * hd))
        else:
            self.pool = np.zeros((num, n_kv, 18 * hd), dtype=np.uint8)
            spread = np.exp(0.5 * rng.standard_normal((n_kv, hd)))
            packed.write(self.pool, rng.standard_normal((num * 16, n_kv, hd)) * spread,
                         rng.standard_normal((num * 16, n_kv, hd)) * spread, np.arange(num * 16))
        self.cfg = _cfg(B, n_q, n_kv, hd, dtype, self.table.shape[1])
        self.q = torch.from_numpy(rng.standard_normal((n, n_q * hd))).cuda().to(_dt(dtype))
        self.max_rows = max(1, max(rows))
        self.d_pool = torch.from_numpy(self.pool).cuda()
        self.d_table, self.d_start, self.d_pos = (torch.from_numpy(x).cuda() for x in (self.table, self.start, self.pos))
        self.ws, self.err = pe.alloc_attend_workspace(self.cfg), _err()
        self.ws.fill_(255)  # its contents do not matter
        self.out = torch.full((n, n_q * hd), 9.0, device="cuda", dtype=_dt(dtype))

    def run(self, q=None, out=None, max_rows=None):
        pe.attend_packed(self.cfg, self.q if q is None else q, self.d_pool, self.d_table, self.d_start, self.d_pos,
                         max_rows or self.max_rows, self.out if out is None else out, self.ws, self.err)

    def want(self, pos=None, start=None):
        return packed.attend(_np(self.q), self.pool, self.table, self.start if start is None else start,
                             self.pos if pos is None else pos, self.n_q)

    def tolerance(self, out, size, depth):
        L = np.maximum(self.pos + 1, 0)[:, None]
        weights = 2 * (self.hd + 8) * U * depth + 2.0 ** -20 + L * U + (2.0 ** -8 if self.dtype == "bf16" else 0)
        return size * (2 * weights + 2 * L * U) + np.abs(out) * (2.0 ** -8 if self.dtype == "bf16" else 2 * U) + 1e-30

    def check(self, got=None, pos=None, start=None, err=0):
        out, size, depth = self.want(pos, start)
        got = _np(self.out if got is None else got)
        assert int(self.err.item()) == err
        lo, hi = self.start[0], self.start[-1]
        far = np.abs(got - out) - self.tolerance(out, size, depth)
        assert np.isfinite(got).all() and far[lo:hi].max() <= 0, (far[lo:hi].max(), np.argwhere(far > 0)[:5])
        assert (got[:lo] == 9).all() and (got[hi:] == 9).all()


SHAPES = {
    # name: (hd, n_q, n_kv, rows, ctx)
    "token-1": (64, 8, 1, [1], [1]),
    "token-16": (64, 64, 8, [1], [16]),
    "token-ragged": (64, 64, 8, [1] * 5, [1, 17, 300, 64, 1023]),
    "token-hd128": (128, 32, 4, [1] * 4, [5, 129, 640, 777]),
    "token-no-groups": (64, 4, 4, [1] * 3, [33, 7, 250]),
    "token-odd-group": (128, 15, 3, [1] * 2, [95, 400]),
    "token-wide-group": (64, 24, 1, [1] * 2, [70, 513]),
    "token-long": (64, 16, 2, [1], [9001]),
    "token-long-hd128": (128, 8, 1, [1, 1], [6007, 40]),
    "two-rows": (64, 32, 4, [2] * 3, [2, 130, 515]),
    "draft-ragged": (64, 64, 8, [14, 7, 11, 8], [14, 900, 77, 1500]),
    "draft-hd128": (128, 32, 4, [9, 14], [350, 2049]),
    "draft-odd-group": (64, 10, 2, [13, 5], [200, 65]),
    "no-rows-somewhere": (64, 16, 2, [0, 3, 0, 0, 2, 0], [1, 40, 1, 1, 333, 1]),
    "chunk": (64, 16, 2, [100, 33], [100, 700]),
    "chunk-hd128": (128, 8, 1, [150], [1000]),
    "chunk-no-groups": (64, 2, 2, [260, 1], [300, 9]),
    "many-sequences": (64, 8, 1, [1] * 300, [1 + 3 * (i % 40) for i in range(300)]),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_attend_matches_the_formula(name, dtype):
    hd, n_q, n_kv, rows, ctx = SHAPES[name]
    a = Att(dtype, hd, n_q, n_kv, rows, ctx, seed=len(name))
    a.run()
    a.check()
    first = a.out.clone()
    a.out.fill_(9.0)
    a.run()  # the workspace's contents and the order of the work change nothing
    assert torch.equal(first, a.out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_attend_over_arbitrary_bytes(hd, rows, dtype):
    a = Att(dtype, hd, 16, 2, [rows, rows], [rows + 19, rows + 401], seed=hd + rows, raw=True)
    a.run()
    a.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 6, 30])
def test_attend_rows_that_see_nothing_and_rows_outside(rows, dtype):
    """Position -1 gives zeros; rows before the first and behind the last sequence stay as they were."""
    a = Att(dtype, 64, 16, 2, [rows, rows, rows], [50 + rows, 300, rows], seed=rows, gap=2, tail=3, empty=[2, 2 + rows])
    a.run()
    a.check()
    assert bool((a.out[2] == 0).all())


@pytest.mark.parametrize("rows,most", [(1, 1), (14, 14), (14, 40)])
def test_attend_strided_rows(rows, most):
    """Queries inside a fused projection's rows, and the output beside them."""
    a = Att("bf16", 64, 16, 2, [rows, max(1, rows - 4)], [100, 300], seed=3)
    w, n = 16 * 64, a.q.shape[0]
    wide = torch.full((n, 3 * w + 8), 9.0, device="cuda", dtype=torch.bfloat16)
    wide[:, w:2 * w] = a.q
    a.run(q=wide[:, w:2 * w], out=wide[:, 2 * w:3 * w], max_rows=most)
    a.check(got=wide[:, 2 * w:3 * w])
    assert bool((wide[:, :w] == 9).all()) and bool((wide[:, 3 * w:] == 9).all())
    assert torch.equal(wide[:, w:2 * w], a.q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 14, 40])
def test_attend_device_checks(rows, dtype):
    ctx = [200 + rows, 400, 90 + rows]
    # a page id outside the pool counts as zero keys and values
    a = Att(dtype, 64, 16, 2, [rows] * 3, ctx, seed=rows)
    for bad in (-1, a.pool.shape[0]):
        a.table[1, 2] = bad
        a.d_table[1, 2] = bad
        a.err.zero_()
        a.run()
        a.check(err=pe.PE_DEV_BAD_PAGE)
    # positions beyond the table, or below -1: zeros for that row
    a = Att(dtype, 64, 16, 2, [rows] * 3, ctx, seed=rows)
    seen = a.pos.copy()
    for bad in (16 * a.table.shape[1], 1 << 30, -2):
        a.d_pos[rows] = bad
        seen[rows] = -1
        a.err.zero_()
        a.run()
        a.check(pos=seen, err=pe.PE_DEV_BAD_POSITION)
    # a sequence with more rows than max_rows, or outside the rows: left as it was, the others are not
    a = Att(dtype, 64, 16, 2, [rows, rows + 1, rows], ctx, seed=rows)
    a.run(max_rows=rows)
    out, size, depth = a.want()
    got = _np(a.out)
    assert int(a.err.item()) == pe.PE_DEV_BAD_ROW
    z = slice(rows, 2 * rows + 1)
    assert (got[z] == 9).all()
    far = np.abs(got - out) - a.tolerance(out, size, depth)
    far[z] = 0
    assert far.max() <= 0
    for bad in (10 * rows + 7, -3):
        a = Att(dtype, 64, 16, 2, [rows] * 3, ctx, seed=rows)
        a.d_start[3] = bad
        a.run()
        assert int(a.err.item()) == pe.PE_DEV_BAD_ROW
        assert bool((a.out[2 * rows:] == 9).all())


def test_attend_refuses_tensors_of_another_kind():
    a = Att("bf16", 64, 16, 2, [2], [40])
    with pytest.raises(ValueError):
        a.run(q=a.q.float())
    with pytest.raises(ValueError):
        a.run(q=a.q[:, ::2])
    with pytest.raises(ValueError):
        a.run(q=a.q.cpu())
    with pytest.raises(ValueError):
        a.run(out=a.out[:1])
    with pytest.raises(pe.PeError):
        a.run(out=a.q)
    with pytest.raises(pe.PeError):
        a.run(max_rows=-1)
    a.ws = a.ws[:-256]
    with pytest.raises(pe.PeError):
        a.run()
    x = torch.zeros(3, 2, 64, device="cuda").bfloat16()
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        pe.pack_kv(a.cfg, x, x, slots.int(), a.d_pool, a.err)
    with pytest.raises(ValueError):
        pe.pack_kv(a.cfg, x[:, :, ::2], x, slots, a.d_pool, a.err)
    with pytest.raises(ValueError):
        pe.unpack_kv(a.cfg, a.d_pool[:, :1], slots, x, x.clone(), a.err)
    # no rows at all: fine
    none = torch.zeros((0, 2, 64), device="cuda").bfloat16()
    pe.pack_kv(a.cfg, none, none, slots[:0], a.d_pool, a.err)
    pe.unpack_kv(a.cfg, a.d_pool, slots[:0], none, none.clone(), a.err)
    assert int(a.err.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_round_of_pack_and_attend_captured_and_replayed(dtype):
    """The operators as a decoder uses them: each round packs its new rows and attends to them, on a
    stream of its own, directly and as a graph that is replayed over changed inputs."""
    B, hd, n_q, n_kv, K = 3, 64, 16, 2, 4
    ctx = [60, 140, 271]
    a = Att(dtype, hd, n_q, n_kv, [K] * B, ctx, seed=11)
    n = B * K
    side = torch.cuda.Stream()
    k, v = (torch.empty((n, n_kv, hd), device="cuda", dtype=_dt(dtype)) for _ in range(2))
    slots = torch.empty(n, dtype=torch.int64, device="cuda")
    rng = np.random.default_rng(5)

    def fill(shift):
        pos = a.pos - 8 + shift  # the rows move on by `shift`
        slot = np.array([a.table[r // K, pos[r] // 16] * 16 + pos[r] % 16 for r in range(n)], dtype=np.int64)
        kk, vv = rng.standard_normal((n, n_kv, hd)), rng.standard_normal((n, n_kv, hd))
        k.copy_(torch.from_numpy(kk))
        v.copy_(torch.from_numpy(vv))
        slots.copy_(torch.from_numpy(slot))
        a.d_pos.copy_(torch.from_numpy(pos))
        a.q.copy_(torch.randn(n, n_q * hd, device="cuda"))
        packed.write(a.pool, _np(k), _np(v), slot)
        return pos

    def once():
        pe.pack_kv(a.cfg, k, v, slots, a.d_pool, a.err)
        a.run()

    pos = fill(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        once()
    side.synchronize()
    a.check(pos=pos)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        once()
    for shift in (4, 8):
        pos = fill(shift)
        a.out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        a.check(pos=pos)


# ----------------------------------------------------------------------------- more of what the calls allow

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_kv,hd,n", [(9, 128, 21), (20, 64, 19), (40, 128, 3), (1, 64, 20011), (16, 128, 2500)])
def test_pack_and_unpack_many_heads_and_rows(dtype, n_kv, hd, n):
    """More heads than a CTA takes at once, numbers of heads that leave lanes over, several rows a lane."""
    rng = np.random.default_rng(n)
    pages = n // 16 + 2
    cfg = _cfg(1, n_kv, n_kv, hd, dtype, pages)
    k, v = (torch.randn(n, n_kv, hd, device="cuda").to(_dt(dtype)) for _ in range(2))
    slots = rng.permutation(pages * 16)[:n].astype(np.int64)
    slots[::7] = -1
    s = torch.from_numpy(slots).cuda()
    pool, err = pe.alloc_packed_pool(cfg, pages), _err()
    pe.pack_kv(cfg, k, v, s, pool, err)
    want = np.zeros(tuple(pool.shape), dtype=np.uint8)
    packed.write(want, _np(k), _np(v), slots)
    assert np.array_equal(pool.cpu().numpy(), want)
    ko, vo = torch.full_like(k, 7), torch.full_like(v, 7)
    pe.unpack_kv(cfg, pool, s, ko, vo, err)
    wk, wv = packed.read(want, np.maximum(slots, 0))
    dead = (slots < 0)[:, None, None]
    assert np.array_equal(_np(ko), np.where(dead, 7, wk)) and np.array_equal(_np(vo), np.where(dead, 7, wv))
    assert int(err.item()) == 0


MORE = {
    # name: (dtype, hd, n_q, n_kv, rows, ctx, max_rows): more tiles than a launch takes, bounds above the rows
    "token-1100-sequences": ("bf16", 64, 8, 1, [1] * 1100, [1 + (7 * i) % 90 for i in range(1100)], 1),
    "f32-1100-sequences": ("f32", 64, 2, 2, [1] * 1100, [1 + (5 * i) % 60 for i in range(1100)], 2),
    "loose-bound": ("bf16", 64, 16, 2, [1, 2, 1, 3] * 20, [40 + 11 * i for i in range(80)], 600),
    "f32-loose-bound": ("f32", 64, 8, 2, [1, 2, 1, 3] * 20, [40 + 11 * i for i in range(80)], 300),
    "chunk-beside-tokens": ("bf16", 128, 8, 2, [1] * 9 + [210] + [1] * 6, [30 + 50 * i for i in range(16)], 210),
    "draft-hd128-odd-group": ("bf16", 128, 9, 3, [13, 8, 1], [700, 64, 65], 13),
    "wide-group": ("bf16", 64, 300, 2, [2, 1], [90, 600], 2),
}


@pytest.mark.parametrize("name", list(MORE))
def test_attend_many_tiles_and_loose_bounds(name):
    dtype, hd, n_q, n_kv, rows, ctx, most = MORE[name]
    ctx = [max(c, r) for c, r in zip(ctx, rows)]
    a = Att(dtype, hd, n_q, n_kv, rows, ctx, seed=len(name))
    a.run(max_rows=most)
    a.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd,n_q,rows", [(64, 8, 1), (64, 16, 15), (128, 8, 33)])
def test_attend_positions_in_any_order(hd, n_q, rows, dtype):
    """Rows of a sequence need not be in the order of their positions, nor next to each other."""
    ctx = [700, 90, 333]
    a = Att(dtype, hd, n_q, 2 if n_q > 8 else 1, [rows] * 3, ctx, seed=rows)
    rng = np.random.default_rng(rows)
    a.pos = np.concatenate([rng.integers(-1, c, rows) for c in ctx]).astype(np.int32)
    a.d_pos = torch.from_numpy(a.pos).cuda()
    a.run()
    a.check()


def test_attend_two_calls_at_once_on_streams_of_their_own():
    """Each call with a workspace of its own: the results are those of one after the other."""
    calls = [Att("bf16", 64, 64, 8, [1] * 6, [1500, 20, 900, 3000, 1, 640], seed=1),
             Att("bf16", 64, 64, 8, [14] * 6, [1500, 20, 900, 3000, 16, 640], seed=2),
             Att("bf16", 128, 32, 4, [90, 100], [1000, 1100], seed=3)]
    alone = []
    for a in calls:
        a.run()
        alone.append(a.out.clone())
        a.out.fill_(9.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for a, s in zip(calls, streams):
            pe.attend_packed(a.cfg, a.q, a.d_pool, a.d_table, a.d_start, a.d_pos, a.max_rows, a.out, a.ws, a.err, stream=s)
    torch.cuda.synchronize()
    for a, want in zip(calls, alone):
        assert torch.equal(a.out, want) and int(a.err.item()) == 0


@pytest.mark.parametrize("rows,dtype", [(1, "bf16"), (9, "bf16"), (2, "f32")])
def test_pages_beyond_32_bits_of_a_large_pool(rows, dtype):
    """A cache whose pages lie beyond 4 GiB of its pool: as the same pages in a small pool, bit for bit."""
    a = Att(dtype, 64, 64, 8, [rows, rows], [900, 333], seed=rows)
    n, num = 2 * rows, a.pool.shape[0]
    big_pages = (1 << 32) // (8 * 18 * 64) + 2 * num  # the last `num` pages start beyond 2^32 bytes
    big = torch.empty((big_pages, 8, 18 * 64), dtype=torch.uint8, device="cuda")
    base = big_pages - num
    big[base:].copy_(a.d_pool)
    k, v = (torch.randn(n, 8, 64, device="cuda").to(_dt(dtype)) for _ in range(2))
    slots = torch.tensor([int(a.table[r // rows, a.pos[r] // 16]) * 16 + int(a.pos[r]) % 16 for r in range(n)],
                         dtype=torch.int64, device="cuda")
    pe.pack_kv(a.cfg, k, v, slots, a.d_pool, a.err)
    pe.pack_kv(a.cfg, k, v, slots + base * 16, big, a.err)
    assert torch.equal(big[base:], a.d_pool)
    a.run()
    table = torch.where(a.d_table >= 0, a.d_table + base, a.d_table)
    out = torch.empty_like(a.out)
    pe.attend_packed(a.cfg, a.q, big, table, a.d_start, a.d_pos, rows, out, a.ws, a.err)
    assert torch.equal(out, a.out)
    back = [torch.empty_like(k) for _ in range(4)]
    pe.unpack_kv(a.cfg, a.d_pool, slots, back[0], back[1], a.err)
    pe.unpack_kv(a.cfg, big, slots + base * 16, back[2], back[3], a.err)
    assert torch.equal(back[0], back[2]) and torch.equal(back[1], back[3]) and int(a.err.item()) == 0


@pytest.mark.parametrize("dtype,hd,n_q,n_kv,spare", [("bf16", 128, 4096, 1, 1), ("bf16", 64, 300, 300, 1),
                                                     ("f32", 64, 1024, 1, 1), ("bf16", 64, 16, 2, 1 << 20),
                                                     ("bf16", 64, 64, 2, 1 << 20)])
def test_attend_many_heads_and_wide_tables(dtype, hd, n_q, n_kv, spare):
    """The most query heads, more kv heads than SMs, and a block table far wider than the positions."""
    a = Att(dtype, hd, n_q, n_kv, [2, 1], [70, 45], seed=n_q, spare=spare)
    a.run()
    a.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 14])
def test_attend_rows_that_are_no_numbers_stay_alone(rows, dtype):
    """NaN and infinite queries spoil their own rows' outputs and no other's."""
    a = Att(dtype, 64, 16, 2, [rows] * 4, [200 + rows, 700, 33 + rows, 1200], seed=rows)
    a.run()
    clean = _np(a.out)
    odd = [0, 2 * rows]  # a row each of the first and the third sequence
    a.q[odd[0], 5] = float("nan")
    a.q[odd[1], 70] = float("inf")
    a.run()
    got = _np(a.out)
    rest = np.setdiff1d(np.arange(4 * rows), odd)
    a.q[odd] = 0
    out, size, depth = a.want()
    tol = a.tolerance(out, size, depth)
    assert np.all(np.abs(got - out)[rest] <= tol[rest]) and np.all(np.abs(clean - out)[rest] <= tol[rest])
    assert int(a.err.item()) == 0
