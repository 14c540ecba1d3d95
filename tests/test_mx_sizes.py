"""Sizes of 4-bit matrices that do not fit 32 bits (no GPU)."""

import pytest

import speculative_decoding_step_gb300 as pe

FAR = [(1 << 32, 64), ((1 << 32) + 5, 64), (5, (1 << 32) + 64), (1 << 31, 64), (-(1 << 32) + 5, 64), (5, -(1 << 32) + 64),
       (1 << 70, 64)]


@pytest.mark.parametrize("n,w", FAR)
def test_sizes_beyond_32_bits_are_out_of_range(n, w):
    assert pe.mx_bytes(n, w) == 0
    with pytest.raises(pe.PeError):
        pe.MxMatrix(n, w, device="cpu")
    with pytest.raises(pe.PeError):
        pe.alloc_linear_mx_workspace(n, w, device="cpu")


def test_sizes_within_are_as_they_were():
    assert pe.mx_bytes(1 << 24, 1 << 20) == 8704 << 30 and pe.mx_bytes(0, 64) == 0 and pe.mx_bytes(129, 129) == 4 * 8704
    assert pe.MxMatrix(0, 64, device="cpu").data.numel() == 0
    assert pe.alloc_linear_mx_workspace(0, 64, device="cpu").numel() == 0
