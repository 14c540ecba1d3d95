"""Packed-cache calls as large as their use: attention whose line of work is divided unevenly between an SM's CTAs, and
the drafter over contexts whose ranges are cut and merged, also two rounds at once.

The measures are those of test_gpu_packed.py and test_gpu_packed_drafter.py (tolerances derived there).
"""

import numpy as np
import pytest
import torch

import test_gpu_packed_drafter as drafter
from oracle import packed
from test_gpu_packed import Att, _np

pytestmark = pytest.mark.gpu


class LongAtt(Att):
    def tolerance(self, out, size, depth, pos):
        """Att's, for the rows at these positions."""
        every, self.pos = self.pos, pos
        tol = super().tolerance(out, size, depth)
        self.pos = every
        return tol


def _lengths(n, lo, hi):
    return [lo + (hi - lo) * (7 * i % n) // n for i in range(n)]


TILES = {
    # name: (hd, n_q, n_kv, rows, ctx): at least 16 units of 64 positions per CTA with two CTAs an SM
    "drafts": (64, 64, 8, [7 + i % 8 for i in range(48)], _lengths(48, 500, 2500)),
    "drafts-hd128": (128, 32, 4, [14 - i % 8 for i in range(48)], _lengths(48, 1100, 2600)),
    "chunks": (64, 64, 8, [301, 17, 190], [3100, 2900, 1200]),
    # more tiles than two CTAs of an SM have room for the line of
    "150-drafts-hd128": (128, 32, 4, [9 - i % 3 for i in range(150)], _lengths(150, 600, 1100)),
    "chunks-hd128": (128, 32, 4, [1000, 1500], [1900, 1500]),
    "750-drafts": (64, 4, 2, [10] * 750, _lengths(750, 700, 1000)),
}


@pytest.mark.parametrize("name", list(TILES))
def test_attend_long_lines(name):
    """Every row against the formula for a few sequences, and every row of the call against itself called twice."""
    hd, n_q, n_kv, rows, ctx = TILES[name]
    a = LongAtt("bf16", hd, n_q, n_kv, rows, ctx, seed=len(name), raw=True)
    a.run()
    got = _np(a.out)
    assert int(a.err.item()) == 0 and np.isfinite(got).all()
    B = len(rows)
    for b in sorted({0, 1, B // 3, B // 2, B - 2, B - 1}):
        z = np.arange(a.start[b], a.start[b + 1])
        if len(z) > 12:  # of a chunk: its first rows, some in its middle, its last
            z = np.concatenate([z[:4], z[len(z) // 2:][:4], z[-4:]])
        pages = -(-ctx[b] // 16)
        out, size, depth = packed.attend(_np(a.q)[z], a.pool[a.table[b, :pages]], np.arange(pages)[None],
                                         np.array([0, len(z)]), a.pos[z], n_q)
        far = np.abs(got[z] - out) - a.tolerance(out, size, depth, a.pos[z])
        assert far.max() <= 0, (b, far.max())
    first = a.out.clone()
    a.out.fill_(9.0)
    a.run()
    assert torch.equal(first, a.out)


LONG = {
    # contexts beyond the tables that keep whole ranges (32 to 96 pages)
    "bf16-hd64-long": drafter._cfg(B=2, K=7, prefix_args=(1600, 1700), seed=72),
    "bf16-hd64-L2-few-rows-long": drafter._cfg(B=2, K=1, n_layers=2, prefix_args=(1300, 1500), seed=73),
    "bf16-hd128-L2-long": drafter._cfg(B=2, K=6, n_q=16, n_kv=2, head_dim=128, d=512, n_layers=2,
                                       prefix_args=(1200, 1300), seed=74),
    "f32-hd64-L2-long": drafter._cfg(dtype="f32", B=2, n_layers=2, prefix_args=(1200, 1400), seed=75),
}
drafter.CASES.update(LONG)


@pytest.mark.parametrize("name", list(LONG))
def test_round_over_a_long_packed_cache_against_oracle(name):
    drafter.test_round_over_a_packed_cache_against_oracle(name)


@pytest.mark.parametrize("name", list(LONG))
def test_step_over_a_long_packed_cache_equals_the_stages_and_its_graph(name):
    drafter.test_step_equals_the_stages_and_its_captured_graph(name)


def test_two_rounds_at_once_on_streams_of_their_own():
    """Rounds of two drafters, each with its caches and workspace: as one after the other."""
    cases = [drafter._setup(LONG[name])[0] for name in ("bf16-hd64-long", "bf16-hd128-L2-long")]
    targets = [torch.zeros((c.cfg.B, c.cfg.K + 1), dtype=torch.int32, device="cuda") for c in cases]
    start = [[p.clone() for p in c.kv.pools] for c in cases]

    def step(c, t):
        R = c.Rd
        c.rd.step(R["prev_tokens"], R["prev_pos"], R["num_accepted"], R["bonus"], R["target_hidden"], t, logits=True)

    want = []
    for c, t in zip(cases, targets):
        step(c, t)
        want.append([c.rd.draft_tokens.clone(), c.rd.logits.clone()] + [p.clone() for p in c.kv.pools])
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        for c, pools in zip(cases, start):
            c.rd.logits.zero_()
            for p, q in zip(c.kv.pools, pools):
                p.copy_(q)
        torch.cuda.synchronize()
        for _ in range(5):
            for c, t, s in zip(cases, targets, streams):
                with torch.cuda.stream(s):
                    step(c, t)
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert int(c.rd.err.item()) == 0
            for x, y in zip([c.rd.draft_tokens, c.rd.logits] + c.kv.pools, w):
                assert torch.equal(x, y)
