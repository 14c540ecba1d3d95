"""Appending rows, without a GPU: outputs over the positions and slots that other rows still read are refused before
anything is launched (placeholder pointers, never dereferenced)."""

import pytest
import torch

import speculative_decoding_step_gb300 as pe
from test_mx_host import _append, _append_packed, _cfg

N = 40  # rows: 320 bytes of slots, 160 of positions for each axis
POS, SLOTS, OUT, CACHE = 1 << 53, 1 << 54, 1 << 55, 1 << 56
REFUSED = 1
LAUNCHED = 4  # as far as the launch, with no device there


@pytest.mark.parametrize("call", [_append, _append_packed])
def test_outputs_over_positions_or_slots_are_refused(call):
    c = _cfg()
    page = 16 * 2 * 64 * 2 if call is _append else pe.packed_page_bytes(c)
    # a cache that begins, lies around or ends there
    for name, at, size in (("pos", POS, 3 * N * 4), ("slots", SLOTS, N * 8)):
        for start in (at, at + size - 16, at - 4 * page + 16, at - page):
            assert call(c, n=N, axes=3, kc=start) == REFUSED, (name, start - at)
    # queries written over either, from the first row or into the last
    row, last = 512 * 2, (N - 1) * 512 * 2
    for at, size in ((POS, 3 * N * 4), (SLOTS, N * 8)):
        for start in (at, at + size - 16, at - row + 16, at - last, at - last - row + 16):
            assert call(c, n=N, axes=3, qo=start) == REFUSED, start - at
            assert call(c, n=N, axes=3, q=start, qo=start) == REFUSED  # in place


@pytest.mark.parametrize("call", [_append, _append_packed])
def test_the_second_cache_is_looked_at_too(call):
    c = _cfg()
    if call is _append:
        assert call(c, n=N, vc=POS) == REFUSED and call(c, n=N, vc=SLOTS) == REFUSED
    else:
        assert call(c, n=N, q=None, qo=None, kc=POS) == REFUSED and call(c, n=N, q=None, qo=None, kc=SLOTS) == REFUSED


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are placeholders: nothing may be launched")
@pytest.mark.parametrize("call", [_append, _append_packed])
def test_outputs_beside_positions_and_slots_are_not_refused(call):
    c = _cfg()
    page = 16 * 2 * 64 * 2 if call is _append else pe.packed_page_bytes(c)
    row = 512 * 2
    for at, size in ((POS, 3 * N * 4), (SLOTS, N * 8)):
        assert call(c, n=N, axes=3, kc=at - 4 * page) == LAUNCHED and call(c, n=N, axes=3, kc=at + size) == LAUNCHED
        assert call(c, n=N, axes=3, qo=at - N * row) == LAUNCHED and call(c, n=N, axes=3, qo=at + size) == LAUNCHED
        # between two rows of queries: a gap of 512 bytes, which takes either
        for k in (0, 7, N - 2):
            assert call(c, n=N, axes=3, qo=at - k * 2 * row - row, qos=2 * 512) == LAUNCHED
            assert call(c, n=N, axes=3, qo=at - k * 2 * row - row + 16, qos=2 * 512) == REFUSED
    assert call(c, n=0, qo=POS, kc=SLOTS) == 0  # no rows
