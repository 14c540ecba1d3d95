"""Caches that append_kv is given as something other than a list of two tensors that are kept."""

import gc

import pytest
import torch

import speculative_decoding_step_gb300 as pe

pytestmark = pytest.mark.gpu


def _case():
    cfg = pe.Config.make(1, 1, 64, 4, 2, 64, 64, 2, 1, 1, "bf16")
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = torch.randn((2, 9, 128), device="cuda", generator=g).bfloat16()
    pos, slots = torch.arange(9, dtype=torch.int32, device="cuda"), torch.arange(9, device="cuda")
    return cfg, k, v, pos, slots, torch.zeros(1, dtype=torch.int32, device="cuda")


class _Pages:
    """Both caches in one tensor; each is a new view when it is asked for, which nobody keeps."""

    def __init__(self, both):
        self.both, self.asked = both, 0

    def __len__(self):
        return 2

    def __getitem__(self, i):
        self.asked += 1
        return self.both[i]


def test_a_sequence_that_makes_its_tensors_when_asked():
    cfg, k, v, pos, slots, err = _case()
    both, want = torch.zeros((2, 2, 1, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    pe.append_kv(cfg, None, k, v, pos, slots, (want[0], want[1]), None, err)
    for _ in range(50):
        both.zero_()
        pages = _Pages(both)
        pe.append_kv(cfg, None, k, v, pos, slots, pages, None, err)
        assert pages.asked == 2 and torch.equal(both, want)
        gc.collect()
    assert int(err.item()) == 0


def test_sequences_that_are_no_pair_are_refused():
    cfg, k, v, pos, slots, err = _case()
    c = torch.zeros((1, 16, 2, 64), dtype=torch.bfloat16, device="cuda")

    class Failing(_Pages):
        def __getitem__(self, i):
            raise KeyError(i)

    for cache in ((c,), (c, c, c), None, 5, {c}, (c, None), ("a", "b")):
        with pytest.raises(ValueError):
            pe.append_kv(cfg, None, k, v, pos, slots, cache, None, err)
    with pytest.raises(KeyError):
        pe.append_kv(cfg, None, k, v, pos, slots, Failing(None), None, err)
