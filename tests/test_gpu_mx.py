"""Microscaled 4-bit matrices on the GPU: quantising, reading back and products against the definition in 64 bits.

Quantising is compared byte for byte and reading back value for value.  A product's tolerance per element is
  width * 2^-23 * sum |x w|    (that many additions in fp32, each off by at most a step, of terms that are exact)
and half a step of the output's type, 2^-8 of it for bf16 and 2^-24 for fp32, with the addition of `add` counted as one
more term.  Where every partial sum is a multiple of a power of two below 2^24 of it, fp32 sums are exact in any order,
and equality is asked for.
"""

import numpy as np
import pytest
import torch

import speculative_decoding_step_gb300 as pe
from oracle import mx

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _np(t):
    return t.detach().double().cpu().numpy()


def _apart(x, dtype, pad=0, off=0):
    """Rows x on the GPU, `pad` elements between them, the first `off` elements into its buffer."""
    n, w = x.shape
    room = torch.full((n * (w + pad) + off + 1,), 7.0, dtype=DT[dtype], device="cuda")
    rows = room[off:off + n * (w + pad)].view(n, w + pad)[:, :w]
    rows.copy_(torch.from_numpy(np.ascontiguousarray(x)))
    return rows


def _wild(rng, n, w):
    """Rows with blocks of zeros, of midpoints, of tiny and of huge entries."""
    x = rng.standard_normal((n, w)) * np.exp(2 * rng.standard_normal((n, 1)))
    mids = np.array([4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 7])
    for r in range(n):
        for b in range(0, w, 32):
            z = slice(b, min(b + 32, w))
            kind = rng.integers(0, 9)
            if kind == 0:
                x[r, z] = 0
            elif kind == 1:
                x[r, z] = np.resize(mids, z.stop - b) * 2.0 ** rng.integers(-100, 100)
            elif kind == 2:
                x[r, z] *= 2.0 ** -125
            elif kind == 3:
                x[r, z] = np.clip(x[r, z], -3, 3) * 2.0 ** 125
            elif kind == 4:
                x[r, z] *= 2.0 ** -145  # denormal in fp32 (and zeros)
    return np.clip(x, -3.3e38, 3.3e38)


SHAPES = [(1, 1), (1, 32), (3, 31), (14, 2880), (130, 33), (8, 257), (257, 128), (129, 1000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (5, 3)])
@pytest.mark.parametrize("n,w", SHAPES)
def test_quantise_and_read_back_match_the_definition(dtype, pad, off, n, w):
    rng = np.random.default_rng(n * 1000 + w)
    x = _apart(_wild(rng, n, w).astype(np.float32), dtype, pad, off)
    before = rng.integers(0, 256, pe.mx_bytes(n, w), dtype=np.uint8)
    m, err = pe.MxMatrix(n, w, data=torch.from_numpy(before).cuda()), _err()
    pe.quantize_mx(x, m, err)
    want = before.copy()
    mx.write(want, _np(x))
    got = m.data.cpu().numpy()
    assert np.array_equal(got, want) and int(err.item()) == 0
    for out_type in ("bf16", "f32"):
        out = _apart(np.full((n, w), 7.0), out_type, pad, off)
        pe.dequantize_mx(m, out)
        assert np.array_equal(_np(out), mx.kept(_np(x)))
        room = torch.as_strided(out, (n * (w + pad) + off + 1,), (1,), 0).clone()
        room[off:off + n * (w + pad)].view(n, w + pad)[:, :w] = 7
        assert bool((room == 7).all())  # nothing between or beside the rows was written


def test_every_fp32_exponent_and_the_neighbours_of_midpoints():
    rows = []
    for k in range(-149, 128):
        for m in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            row = np.zeros(32)
            with np.errstate(over="ignore", under="ignore"):
                top = np.float32(np.ldexp(1.0, k))
                mid = np.float32(np.ldexp(m / 4, k))
                row[:4] = [top, mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(np.inf))]
            row[4:8] = -row[:4]
            rows.append(np.where(np.isfinite(row), row, 0))
    x = torch.from_numpy(np.array(rows, dtype=np.float32)).cuda()
    m, err = pe.MxMatrix(len(rows), 32), _err()
    pe.quantize_mx(x, m, err)
    out = torch.empty_like(x)
    pe.dequantize_mx(m, out)
    assert np.array_equal(_np(out), mx.kept(_np(x))) and int(err.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantise_reports_and_keeps_numbers(dtype):
    x = torch.randn(5, 100, device="cuda").to(DT[dtype])
    x[1, 3], x[2, 40], x[2, 41], x[4, 99] = float("nan"), float("inf"), float("-inf"), float("nan")
    x[3, 32:64] = float("inf")
    m, err = pe.MxMatrix(5, 100), _err()
    m.data.zero_()
    pe.quantize_mx(x, m, err)
    want = np.zeros(m.data.numel(), np.uint8)
    mx.write(want, _np(x))
    assert np.array_equal(m.data.cpu().numpy(), want) and int(err.item()) == pe.PE_DEV_NONFINITE


def test_no_rows():
    err = _err()
    m = pe.MxMatrix(0, 64)
    w = pe.MxMatrix(3, 64)
    e = torch.empty((0, 64), device="cuda")
    y = torch.empty((0, 3), device="cuda")
    pe.quantize_mx(e, m, err)
    pe.dequantize_mx(m, e)
    pe.matmul_mx(m, w, y, err)
    pe.linear_mx(e, w, y, pe.alloc_linear_mx_workspace(0, 64), err)


# ----------------------------------------------------------------------------- products

def _product_case(rng, n, m, w, exact):
    """Rows and weights as fp32; exact: every entry is kept as it is and every sum is exact."""
    if exact:
        out = []
        for rows in (n, m):
            v = mx.LEVELS[rng.integers(0, 8, (rows, w))] * rng.choice([-1.0, 1.0], (rows, w))
            v[:, ::32] = 4.0  # so a block's scale is 1
            e = np.repeat(rng.integers(0, 3, (rows, -(-w // 32))), 32, axis=1)[:, :w]
            out.append(v * 2.0 ** e)
        return out
    return [rng.standard_normal((n, w)) * np.exp(0.5 * rng.standard_normal(w)), 0.02 * rng.standard_normal((m, w))]


def _mx(x, garbage=255):
    """A matrix of rows x whose unused bytes are `garbage` (255: NaN scales)."""
    m = pe.MxMatrix(*x.shape)
    m.data.fill_(garbage)
    err = _err()
    pe.quantize_mx(torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda(), m, err)
    assert int(err.item()) == 0
    return m


def _compare(y, x, w, add, out):
    xk, wk = mx.kept(x.astype(np.float32)), mx.kept(w.astype(np.float32))
    want, size = xk @ wk.T, np.abs(xk) @ np.abs(wk).T
    terms = x.shape[1]
    if add is not None:
        want, size, terms = want + add, size + np.abs(add), terms + 1
    tol = terms * 2.0 ** -23 * size
    tol = tol + HALF[out] * (np.abs(want) + tol)
    bad = np.abs(y - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], y[bad][:5], want[bad][:5])


PRODUCTS = [(1, 1, 1), (1, 128, 128), (1, 130, 33), (7, 300, 256), (8, 768, 256), (14, 1000, 2880), (16, 129, 31),
            (17, 257, 544), (33, 640, 1000), (64, 127, 96), (100, 2880, 7680), (128, 256, 384), (129, 200, 160),
            (200, 1, 500), (257, 513, 129), (300, 1500, 640), (640, 384, 2880), (1000, 700, 257)]


@pytest.mark.parametrize("n,m,w", PRODUCTS)
@pytest.mark.parametrize("out,add", [("bf16", False), ("f32", False), ("f32", True), ("bf16", True)])
def test_product_against_64_bits(n, m, w, out, add):
    rng = np.random.default_rng(n * 7 + m * 3 + w)
    x, wt = _product_case(rng, n, m, w, False)
    y = _apart(np.full((n, m), np.nan), out, 5 if add else 0, 3 if add else 0)
    a = _apart(rng.standard_normal((n, m)), out, 1, 1) if add else None
    err = _err()
    pe.matmul_mx(_mx(x), _mx(wt), y, err, add=a)
    assert int(err.item()) == 0
    _compare(_np(y), x, wt, _np(a) if add else None, out)
    if add:  # rows apart: nothing between them was written
        room = torch.as_strided(y, (n, m + 5), (m + 5, 1), 3)
        assert bool((room[:-1, m:] == 7).all())


@pytest.mark.parametrize("n,m,w", [(1, 200, 512), (5, 129, 1000), (14, 300, 1777), (130, 257, 640), (300, 128, 96),
                                   (513, 300, 257)])
def test_product_is_exact_where_sums_are(n, m, w):
    rng = np.random.default_rng(n + m + w)
    x, wt = _product_case(rng, n, m, w, True)
    y, err = torch.full((n, m), float("nan"), device="cuda"), _err()
    pe.matmul_mx(_mx(x), _mx(wt), y, err)
    assert np.array_equal(mx.kept(x), x) and np.array_equal(_np(y), x @ wt.T) and int(err.item()) == 0


# Tiles that two, four or eight CTAs share along k, with columns that do not divide evenly among them; far more rows than
# anything else, one record of weights
@pytest.mark.parametrize("n,m,w", [(16, 128, 8192), (7, 5000, 8000), (9, 2100, 5000), (64, 700, 6000), (50, 4500, 8192),
                                   (100, 130, 8100), (128, 2000, 8192), (33, 129, 4097), (400000, 100, 100)])
@pytest.mark.parametrize("out,add", [("f32", False), ("f32", True)])
def test_product_of_shared_tiles_is_exact_where_sums_are(n, m, w, out, add):
    rng = np.random.default_rng(n + m + w)
    small = rng.choice([-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5, 2.0, 4.0], size=(n, w))
    small[:, ::32] = 4.0                                       # every block's scale is 1
    wt = rng.choice([-1.0, -0.5, 0.0, 0.5, 1.0, 4.0], size=(m, w))
    wt[:, ::32] = -4.0
    y = torch.full((n, m), float("nan"), device="cuda")
    a = torch.from_numpy(rng.integers(-64, 64, (n, m)).astype(np.float32)).cuda() if add else None
    err = _err()
    pe.matmul_mx(_mx(small), _mx(wt), y, err, add=a)
    want = small.astype(np.float32) @ wt.T.astype(np.float32)  # multiples of 1/4 below 2^18: exact in fp32 in any order
    assert np.array_equal(y.cpu().numpy(), want + a.cpu().numpy() if add else want) and int(err.item()) == 0


# many rows, from one unit of 256 x 256 a pair of CTAs to several each, with odd numbers of 128-row blocks on either side
MANY = [(2000, 2000, 257), (1300, 5200, 100), (3000, 3000, 300), (4099, 6000, 200), (2900, 7900, 1000)]


@pytest.mark.parametrize("n,m,w", MANY)
@pytest.mark.parametrize("exact,out,add", [(True, "f32", False), (False, "bf16", False), (False, "f32", True)])
def test_product_of_many_rows(n, m, w, exact, out, add):
    rng = np.random.default_rng(n + m + w)
    x, wt = _product_case(rng, n, m, w, exact)
    y = _apart(np.full((n, m), np.nan), out, 3 if add else 0)
    a = torch.randn((n, m), device="cuda").to(DT[out]) if add else None
    err = _err()
    pe.matmul_mx(_mx(x), _mx(wt), y, err, add=a)
    assert int(err.item()) == 0
    if exact:
        assert np.array_equal(_np(y), x @ wt.T)
    else:
        _compare(_np(y), x, wt, _np(a) if add else None, out)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("n,m,w,pad", [(1, 129, 33, 0), (7, 768, 256, 8), (14, 640, 2880, 0), (16, 300, 257, 3),
                                       (17, 128, 96, 0), (64, 500, 1000, 24), (200, 300, 640, 0)])
def test_linear_is_the_product_of_its_quantised_rows(dtype, out, n, m, w, pad):
    rng = np.random.default_rng(n + 10 * m + w)
    x, wt = _product_case(rng, n, m, w, False)
    rows, wm, err = _apart(x, dtype, pad), _mx(wt), _err()
    ws = pe.alloc_linear_mx_workspace(n, w)
    ws.fill_(255)
    y = torch.full((n, m), float("nan"), dtype=DT[out], device="cuda")
    pe.linear_mx(rows, wm, y, ws, err)
    _compare(_np(y), _np(rows), wt, None, out)
    # in place on a residual stream
    z = torch.randn((n, m), device="cuda").to(DT[out])
    before = _np(z)
    pe.linear_mx(rows, wm, z, ws, err, add=z)
    _compare(_np(z), _np(rows), wt, before, out)
    assert int(err.item()) == 0


def test_linear_reports_entries_that_are_no_numbers():
    x = torch.randn(9, 300, device="cuda")
    x[4, 200] = float("nan")
    w, err = _mx(np.random.default_rng(0).standard_normal((140, 300))), _err()
    y = torch.empty((9, 140), device="cuda")
    pe.linear_mx(x, w, y, pe.alloc_linear_mx_workspace(9, 300), err)
    assert int(err.item()) == pe.PE_DEV_NONFINITE
    x[4, 200] = 0
    z, err = torch.empty_like(y), _err()
    pe.linear_mx(x, w, z, pe.alloc_linear_mx_workspace(9, 300), err)
    assert torch.equal(y, z) and int(err.item()) == 0


def test_repeated_products_are_the_same_bits():
    rng = np.random.default_rng(5)
    for n, m, w in ((7, 3000, 2880), (300, 1000, 1000)):
        x, wt = _product_case(rng, n, m, w, False)
        xm, wm, err = _mx(x), _mx(wt), _err()
        ys = [torch.empty((n, m), device="cuda") for _ in range(3)]
        for y in ys:
            pe.matmul_mx(xm, wm, y, err)
        assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_rows_do_not_depend_on_their_neighbours_bytes():
    """The first rows of a matrix, and weights from a multiple of 128 rows on, are matrices."""
    rng = np.random.default_rng(6)
    x, wt = _product_case(rng, 40, 400, 700, False)
    xm, wm, err = _mx(x), _mx(wt), _err()
    y = torch.empty((11, 400), device="cuda")
    pe.matmul_mx(xm.first(11), wm, y, err)
    _compare(_np(y), x[:11], wt, None, "f32")
    part = pe.MxMatrix(144, 700, data=wm.data[pe.mx_bytes(256, 700):])
    z = torch.empty((40, 144), device="cuda")
    pe.matmul_mx(xm, part, z, err)
    _compare(_np(z), x, wt[256:], None, "f32")


def test_the_largest_sizes():
    err = _err()
    rows = 1 << 24                                             # one entry a row: each is kept as the block's largest
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.tensor([0.0, 4.0, -5.0, 6.0, 7.0, 96.0], device="cuda")[torch.randint(0, 6, (rows, 1), device="cuda",
                                                                                   generator=g)]
    m = pe.MxMatrix(rows, 1)
    pe.quantize_mx(x, m, err)
    back = torch.empty_like(x)
    pe.dequantize_mx(m, back)
    kept = torch.where(x == -5.0, -4.0, torch.where(x == 7.0, 6.0, x))  # -5 and 7 lie between 4 and 6, and 6 and 8
    assert torch.equal(back, kept)
    y = torch.empty((rows, 1), device="cuda")
    pe.matmul_mx(m, _mx(np.array([[3.0]])), y, err)
    assert torch.equal(y, 3 * kept)
    del m, x, back, kept, y
    width = 1 << 20
    rng = np.random.default_rng(9)
    x, wt = rng.choice([-1.0, 0.0, 1.0], (3, width)), rng.choice([-0.5, 0.5, 1.0], (5, width))
    x[:, ::32], wt[:, ::32] = 4.0, 4.0
    y = torch.empty((3, 5), device="cuda")
    pe.matmul_mx(_mx(x), _mx(wt), y, err)                      # multiples of 1/2 below 2^21: exact in any order
    assert np.array_equal(_np(y), x @ wt.T) and int(err.item()) == 0


def test_a_matrix_times_itself():
    rng = np.random.default_rng(12)
    for n, w in ((20, 300), (200, 1000)):
        x, _ = _product_case(rng, n, 1, w, True)
        m, y, err = _mx(x), torch.empty((n, n), device="cuda"), _err()
        pe.matmul_mx(m, m, y, err)
        assert np.array_equal(_np(y), x @ x.T) and int(err.item()) == 0


def test_products_on_two_streams_at_once():
    """Kept rows, tiles of a CTA, of a cluster and of a pair, each beside the others, on the same matrices."""
    err = _err()
    g = torch.Generator(device="cuda").manual_seed(8)
    cases = []
    for n, m, w in ((8, 20000, 2880), (128, 4000, 2000), (100, 300, 8192), (1000, 8192, 2048)):
        x, wm = pe.MxMatrix(n, w), pe.MxMatrix(m, w)
        pe.quantize_mx(torch.randn(n, w, device="cuda", generator=g), x, err)
        pe.quantize_mx(torch.randn(m, w, device="cuda", generator=g), wm, err)
        want = torch.empty((n, m), device="cuda")
        pe.matmul_mx(x, wm, want, err)
        cases.append((x, wm, want))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(24):
        for k, s in enumerate(streams):
            x, wm, want = cases[(i + k) % len(cases)]
            with torch.cuda.stream(s):
                y = torch.empty_like(want)
            pe.matmul_mx(x, wm, y, err, stream=s)
            got.append((y, want))
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and all(torch.equal(y, want) for y, want in got)


def test_scale_bytes_that_stand_for_nan_and_extremes():
    rng = np.random.default_rng(8)
    x, wt = _product_case(rng, 3, 130, 160, True)
    xm, wm, err = _mx(x, 0), _mx(wt, 0), _err()
    wm.data[2 * mx.RECORD + mx.scale_at(1, 0)] = 255  # row 129: the second 128 rows, their first piece
    y = torch.empty((3, 130), device="cuda")
    pe.matmul_mx(xm, wm, y, err)
    got = _np(y)
    assert np.isnan(got[:, 129]).all() and np.array_equal(got[:, :129], (x @ wt.T)[:, :129])
    # scales of 2^100 and 2^-100 meet
    wt2, x2 = wt * 2.0 ** 100, x * 2.0 ** -100
    pe.matmul_mx(_mx(x2), _mx(wt2), y, err)
    assert np.array_equal(_np(y), x @ wt.T)


def test_products_on_another_stream_and_captured():
    rng = np.random.default_rng(9)
    n, m, w = 14, 900, 1000
    x, wt = _product_case(rng, n, m, w, False)
    wm, err = _mx(wt), _err()
    xs = torch.from_numpy(x.astype(np.float32)).cuda()
    ws = pe.alloc_linear_mx_workspace(n, w)
    y = torch.empty((n, m), device="cuda")
    want = torch.empty_like(y)
    pe.linear_mx(xs, wm, want, ws, err)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pe.linear_mx(xs, wm, y, ws, err, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pe.linear_mx(xs, wm, y, ws, err)
    for k in range(3):
        xs.copy_(torch.from_numpy((x * (k + 1)).astype(np.float32)))
        pe.linear_mx(xs, wm, want, ws, err)
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert int(err.item()) == 0


@pytest.mark.parametrize("n, m, w, stage", [(8, 768, 256, 0), (100, 256, 1024, 0), (100, 20000, 2560, 1),
                                            (1000, 12288, 2048, 0), (1000, 12288, 2048, 3), (1000, 12288, 2048, 6)])
def test_a_wait_that_runs_out_ends_the_call_and_the_next_one_passes(n, m, w, stage):
    err = _err()
    g = torch.Generator(device="cuda").manual_seed(n + m)
    x = torch.randn(n, w, device="cuda", generator=g)
    wm = pe.MxMatrix(m, w)
    pe.quantize_mx(torch.randn(m, w, device="cuda", generator=g), wm, err)
    ws = pe.alloc_linear_mx_workspace(n, w)
    want, y = torch.empty((n, m), device="cuda"), torch.empty((n, m), device="cuda")
    pe.linear_mx(x, wm, want, ws, err)
    assert int(err.item()) == 0
    pe.set_wait_limit_ns(1_000_000)
    try:
        pe.skip_pipeline_stage_for_test(stage)
        pe.linear_mx(x, wm, y, ws, err)
        torch.cuda.synchronize()
    finally:
        pe.skip_pipeline_stage_for_test(-1)
        pe.set_wait_limit_ns(0)
    assert int(err.item()) == pe.PE_DEV_TIMEOUT
    err.zero_()
    pe.linear_mx(x, wm, y, ws, err)
    assert int(err.item()) == 0 and torch.equal(y, want)


def test_python_refusals():
    err = _err()
    w, y = pe.MxMatrix(5, 64), torch.empty((3, 5), device="cuda")
    x = torch.randn(3, 64, device="cuda")
    ws = pe.alloc_linear_mx_workspace(3, 64)
    with pytest.raises(ValueError):
        pe.quantize_mx(x.half(), pe.MxMatrix(3, 64), err)
    with pytest.raises(ValueError):
        pe.quantize_mx(x, pe.MxMatrix(4, 64), err)
    with pytest.raises(ValueError):
        pe.quantize_mx(x.cpu(), pe.MxMatrix(3, 64), err)
    with pytest.raises(ValueError):
        pe.quantize_mx(torch.randn(64, 3, device="cuda").t(), pe.MxMatrix(3, 64), err)
    with pytest.raises(ValueError):
        pe.matmul_mx(pe.MxMatrix(3, 96), w, y, err)
    with pytest.raises(ValueError):
        pe.linear_mx(x, w, y, ws, err, add=y.bfloat16())
    with pytest.raises(ValueError):
        pe.linear_mx(x, w, torch.empty((3, 6), device="cuda"), ws, err)
    with pytest.raises(pe.PeError):
        pe.linear_mx(x, w, y, ws[:256], err)
    with pytest.raises(pe.PeError):
        pe.MxMatrix(3, 0)
    with pytest.raises(ValueError):
        pe.MxMatrix(3, 64, data=torch.empty(100, dtype=torch.uint8, device="cuda"))
