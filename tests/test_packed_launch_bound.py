"""The number of launches that attend_packed's bounds may ask for, as pe.h states it (no GPU: placeholder pointers, and
calls that are refused or, with no device to launch on, fail)."""

import pytest
import torch

import speculative_decoding_step_gb300 as pe
from test_packed_host import _attend, _cfg


def _launches(c, max_rows):
    vectors = max_rows * (c.n_q // c.n_kv)
    tiles_of = 128 if c.dtype == 1 and vectors > 16 else 8 if vectors <= 8 else 16
    units = -(-c.max_pages_per_seq // (4 if tiles_of == 128 else 2)) + (6 if tiles_of == 128 else 1)
    per_launch = min(1024, max(1, (2 ** 31 - 1) // (c.n_kv * units)))
    return -(-c.B * -(-vectors // tiles_of) // per_launch)


CASES = {
    # name: (config, max_rows): B is the largest of 4096 launches
    "tokens-widest-tables": (dict(n_q=64, n_kv=64, max_pages_per_seq=1 << 24, B=3 * 4096), 1),
    "f32-16-vectors-wide-tables": (dict(n_q=64, n_kv=64, max_pages_per_seq=1 << 24, B=3 * 2048, dtype="f32"), 32),
    "tiles-widest-tables": (dict(n_q=64, n_kv=64, max_pages_per_seq=1 << 24, B=7 * 4096), 128),
    "tiles": (dict(B=4096, max_pages_per_seq=9), 128 * 1024 // 4),
    "tokens-of-8": (dict(n_q=4096, n_kv=2, B=64, max_pages_per_seq=9, dtype="f32"), 512),
}


@pytest.mark.parametrize("name", list(CASES))
def test_bounds_of_more_than_4096_launches_are_refused(name):
    kw, most = CASES[name]
    n = max(most, 1)
    at, above = _cfg(**kw), _cfg(**dict(kw, B=kw["B"] + 1))
    full, w = pe.attend_workspace_bytes(at), at.n_q * 64
    call = lambda c: _attend(c, qs=w, os=w, n=n, most=most, ws_bytes=full)  # noqa: E731
    assert _launches(at, most) == 4096 and _launches(above, most) > 4096
    assert call(above) == 2
    if not torch.cuda.is_available():
        assert call(at) == 4  # goes as far as its launch
