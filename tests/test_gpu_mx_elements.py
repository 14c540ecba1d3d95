"""Products of 4-bit matrices: every element is written, and is a number.

Outputs start as NaN and unused bytes of the matrices as scales that are no numbers, so an element that was left out, or that
something beside its operands reached, is NaN.  A comparison that asks whether a difference is beyond its tolerance passes
those; here each difference has to be within it (_within, which is tested without a GPU).  The tolerance is the one that
test_gpu_mx.py derives: an fp32 step per addition of exact terms, and half a step of the output's type.  Where sums are exact
a bf16 output is the sum rounded once, and equality is asked for.
"""

import numpy as np
import pytest
import torch

import speculative_decoding_step_gb300 as pe
from oracle import mx
from test_gpu_mx import DT, HALF, MANY, PRODUCTS, _apart, _err, _mx, _np, _product_case

gpu = pytest.mark.gpu


def _within(got, want, tol):
    good = np.abs(got - want) <= tol
    assert good.all(), (int((~good).sum()), np.argwhere(~good)[:5], got[~good][:5], want[~good][:5])


def _check(y, x, w, add, out):
    xk, wk = mx.kept(x.astype(np.float32)), mx.kept(w.astype(np.float32))
    want, size, terms = xk @ wk.T, np.abs(xk) @ np.abs(wk).T, x.shape[1]
    if add is not None:
        want, size, terms = want + add, size + np.abs(add), terms + 1
    tol = terms * 2.0 ** -23 * size
    _within(y, want, tol + HALF[out] * (np.abs(want) + tol))


def _rounded(sums, out):
    """Sums that fp32 holds exactly, rounded once to the output's type."""
    assert np.array_equal(sums.astype(np.float32), sums)
    return torch.from_numpy(sums.astype(np.float32)).to(DT[out]).double().numpy()


@pytest.mark.parametrize("bad", [np.nan, np.inf, 2.5])
def test_the_comparison_fails_where_one_element_is_off(bad):
    want = np.ones((3, 4))
    _within(want + 0.5, want, np.full((3, 4), 0.5))
    got = want.copy()
    got[1, 2] = bad
    with pytest.raises(AssertionError):
        _within(got, want, np.ones((3, 4)))
    got[:] = bad
    with pytest.raises(AssertionError):
        _within(got, want, np.ones((3, 4)))


@gpu
@pytest.mark.parametrize("n,m,w", PRODUCTS)
@pytest.mark.parametrize("out,add", [("bf16", False), ("f32", False), ("f32", True), ("bf16", True)])
def test_every_element_of_a_product(n, m, w, out, add):
    rng = np.random.default_rng(n * 7 + m * 3 + w + 1)
    x, wt = _product_case(rng, n, m, w, False)
    y = _apart(np.full((n, m), np.nan), out, 5 if add else 0, 3 if add else 0)
    a = _apart(rng.standard_normal((n, m)), out, 1, 1) if add else None
    err = _err()
    pe.matmul_mx(_mx(x), _mx(wt), y, err, add=a)
    assert int(err.item()) == 0
    _check(_np(y), x, wt, _np(a) if add else None, out)


EXACT = [(1, 200, 512), (14, 300, 1777), (64, 129, 1000), (100, 300, 640), (130, 257, 640), (300, 1500, 96),
         (7, 5000, 8000), (100, 130, 8100), (33, 129, 4097)] + MANY


@gpu
@pytest.mark.parametrize("n,m,w", EXACT)
@pytest.mark.parametrize("out,add", [("bf16", False), ("bf16", True), ("f32", True)])
def test_exact_sums_are_rounded_once(n, m, w, out, add):
    """One CTA's tiles, a cluster's and a pair's.  Entries of one block are at most 4 times a power of two up to 4."""
    rng = np.random.default_rng(n + m + w + 2)
    x = rng.choice([-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5, 2.0, 4.0], size=(n, w))
    wt = rng.choice([-1.0, -0.5, 0.0, 0.5, 1.0, 4.0], size=(m, w))
    x[:, ::32], wt[:, ::32] = 4.0, -4.0                    # every block's scale is 1, so every entry is kept
    y = _apart(np.full((n, m), np.nan), out, 3 if add else 0)
    a = torch.from_numpy(rng.integers(-64, 64, (n, m)).astype(np.float32)).cuda().to(DT[out]) if add else None
    err = _err()
    pe.matmul_mx(_mx(x), _mx(wt), y, err, add=a)
    sums = (x.astype(np.float32) @ wt.T.astype(np.float32)).astype(np.float64)  # multiples of 1/4 below 2^18: exact
    assert int(err.item()) == 0 and np.array_equal(_np(y), _rounded(sums + _np(a) if add else sums, out))


@gpu
@pytest.mark.parametrize("n,m,w", MANY)
@pytest.mark.parametrize("out,add", [("bf16", False), ("f32", True)])
def test_every_element_of_a_product_of_many_rows(n, m, w, out, add):
    rng = np.random.default_rng(n + m + w + 3)
    x, wt = _product_case(rng, n, m, w, False)
    y = _apart(np.full((n, m), np.nan), out, 3 if add else 0)
    a = torch.randn((n, m), device="cuda").to(DT[out]) if add else None
    err = _err()
    pe.matmul_mx(_mx(x), _mx(wt), y, err, add=a)
    assert int(err.item()) == 0
    _check(_np(y), x, wt, _np(a) if add else None, out)


@gpu
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("n,m,w,pad", [(1, 129, 33, 0), (7, 768, 256, 8), (14, 640, 2880, 0), (16, 300, 257, 3),
                                       (17, 128, 96, 0), (64, 500, 1000, 24), (200, 300, 640, 0), (12, 257, 6000, 0),
                                       (1100, 2500, 384, 0)])
def test_every_element_of_linear(dtype, out, n, m, w, pad):
    rng = np.random.default_rng(n + 10 * m + w + 4)
    x, wt = _product_case(rng, n, m, w, False)
    rows, wm, err = _apart(x, dtype, pad), _mx(wt), _err()
    ws = pe.alloc_linear_mx_workspace(n, w)
    ws.fill_(255)
    y = torch.full((n, m), float("nan"), dtype=DT[out], device="cuda")
    pe.linear_mx(rows, wm, y, ws, err)
    _check(_np(y), _np(rows), wt, None, out)
    z = torch.randn((n, m), device="cuda").to(DT[out])
    before = _np(z)
    pe.linear_mx(rows, wm, z, ws, err, add=z)
    _check(_np(z), _np(rows), wt, before, out)
    assert int(err.item()) == 0


@gpu
def test_every_element_beside_rows_of_other_bytes():
    rng = np.random.default_rng(6)
    x, wt = _product_case(rng, 40, 400, 700, False)
    xm, wm, err = _mx(x), _mx(wt), _err()
    y = torch.full((11, 400), float("nan"), device="cuda")
    pe.matmul_mx(xm.first(11), wm, y, err)
    _check(_np(y), x[:11], wt, None, "f32")
    part = pe.MxMatrix(144, 700, data=wm.data[pe.mx_bytes(256, 700):])
    z = torch.full((40, 144), float("nan"), device="cuda")
    pe.matmul_mx(xm, part, z, err)
    _check(_np(z), x, wt[256:], None, "f32")
    assert int(err.item()) == 0


@gpu
def test_more_outputs_than_32_bits_count():
    """2.15e9 elements of y: a one-block width, so that element (r, f) is the product of two small numbers."""
    n, m = 16500, 130200
    assert n * m > 1 << 31
    err = _err()
    g = torch.Generator(device="cuda").manual_seed(2)
    values = torch.tensor([-4.0, -2.0, -1.0, 1.0, 2.0, 4.0], device="cuda")
    sides = [values[torch.randint(0, 6, (k, 1), device="cuda", generator=g)] for k in (n, m)]
    x, w = pe.MxMatrix(n, 1), pe.MxMatrix(m, 1)
    for rows, matrix in zip(sides, (x, w)):
        pe.quantize_mx(rows, matrix, err)
    y = torch.full((n, m), float("nan"), dtype=torch.bfloat16, device="cuda")
    pe.matmul_mx(x, w, y, err)
    want = sides[1].bfloat16().view(1, m)
    for r in range(0, n, 1500):  # products of powers of two: exact
        part = sides[0][r:r + 1500].bfloat16()
        assert torch.equal(y[r:r + 1500], part * want)
    assert int(err.item()) == 0
