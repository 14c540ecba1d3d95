"""Queries of attend_packed that are no numbers: a query head with a NaN or infinite entry gets NaN in every output
entry, whether one CTA finishes its range or several share it, and changes no other head's; where its row sees nothing it
gets zeros.

The other heads are held to the tolerance of test_gpu_packed.py (its derivation stands there).
"""

import numpy as np
import pytest
import torch

import speculative_decoding_step_gb300 as pe
from oracle import packed
from test_gpu_packed import Att, _np

pytestmark = pytest.mark.gpu

CONTEXTS = {
    # tables of at most 32 pages: whole ranges
    "short-table": ([400, 300, 33, 480], 1),
    # the same positions, and longer ones, under a table too wide for that: ranges cut between CTAs, and a merge
    "wide-table": ([400, 300, 33, 480], 300),
    "long": ([1500, 700, 33, 2900], 1),
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [1, 2, 14])
@pytest.mark.parametrize("where", list(CONTEXTS))
def test_attend_queries_that_are_no_numbers_give_nan_and_stay_alone(where, rows, hd, dtype):
    ctx, spare = CONTEXTS[where]
    n_q, n_kv, n = 16, 2, 4 * rows
    unseeing = 2 * rows  # the third sequence's first row
    a = Att(dtype, hd, n_q, n_kv, [rows] * 4, ctx, seed=rows + hd, spare=spare, empty=[unseeing])
    # keys all above zero, so that an infinite entry makes every score infinite and of its sign
    rng = np.random.default_rng(rows)
    shape = (a.pool.shape[0] * 16, n_kv, hd)
    packed.write(a.pool, 1 + np.abs(rng.standard_normal(shape)), rng.standard_normal(shape), np.arange(shape[0]))
    a.d_pool.copy_(torch.from_numpy(a.pool))
    odd = {(0, 0): "nan", (0, 1): "inf", (0, 2): "-inf", (0, 9): "nan", (rows, 15): "-inf", (n - 1, 3): "nan",
           (n - 1, 4): "-inf", (n - 1, 12): "inf", (unseeing, 0): "nan", (unseeing, 8): "inf"}
    out, size, depth = a.want()
    tol = a.tolerance(out, size, depth)
    q = a.q.clone()
    for i, ((r, h), kind) in enumerate(odd.items()):
        q[r, h * hd + 7 * i % hd] = float(kind)
    a.run(q=q)
    got = _np(a.out)
    assert int(a.err.item()) == 0
    for r, h in odd:
        z = slice(h * hd, (h + 1) * hd)
        assert (got[r, z] == 0).all() if r == unseeing else np.isnan(got[r, z]).all(), (r, h, odd[r, h], got[r, z][:4])
        got[r, z] = out[r, z]
    assert np.all(np.abs(got - out) <= tol)
