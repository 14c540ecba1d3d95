"""Microscaled 4-bit matrices and appending without a GPU: the format's definition, and what the calls refuse before
anything is launched (placeholder pointers, never dereferenced: every call here stops at a check or has no rows)."""

import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_step_gb300 as pe
from oracle import mx

AT = 1 << 40
NULL = ctypes.c_void_p(None)


def _p(x=AT):
    return ctypes.c_void_p(x)


# ----------------------------------------------------------------------------- the format

def test_every_byte_of_a_record_is_used_once():
    seen = np.zeros(mx.RECORD, int)
    for r in range(128):
        for b in range(4):
            seen[mx.scale_at(r, b)] += 1
            seen[mx.code_at(r, b):mx.code_at(r, b) + 16] += 1
    assert (seen == 1).all()


def test_first_rows_are_one_run_of_bytes():
    for n in (8, 16, 64, 128):
        assert max(mx.code_at(r, b) + 16 for r in range(n) for b in range(4)) == 512 + 64 * n


def test_kept_values_by_hand():
    x = np.zeros((1, 32))
    x[0, :16] = [4, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 5.1, 7.9, -0.75, -2.5, -5.1, 0.1, -0.1]
    want = [4, 0, 0.5, 1, 1, 2, 2, 4, 4, 6, 6, -1, -2, -6, 0, 0]
    assert np.array_equal(mx.kept(x)[0, :16], want)
    for k in (-120, -3, 5, 120):
        assert np.array_equal(mx.kept(x * 2.0 ** k)[0, :16], np.array(want) * 2.0 ** k)
    assert np.array_equal(mx.kept(np.full((1, 3), 2.0 ** -149)), np.zeros((1, 3)))
    assert mx.quantise(np.zeros((2, 40)))[1].max() == 0


def test_kept_values_are_exact_in_bf16_and_near():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((60, 97)) * np.exp(3 * rng.standard_normal((60, 1)))
    y = mx.kept(x)
    assert np.array_equal(torch.from_numpy(y).bfloat16().double().numpy(), y)
    top = np.abs(mx._blocks(x)).max(-1)
    unit = 2.0 ** (np.floor(np.log2(top)) - 2)
    err = np.abs(mx._blocks(x) - mx._blocks(y)).max(-1)
    assert (err <= 2 * unit).all()  # half a step of 2, or what lies beyond 6 of 8
    assert np.array_equal(mx.kept(y), y)  # what is kept is kept again


def test_sizes():
    assert pe.mx_bytes(1, 1) == 8704 and pe.mx_bytes(128, 128) == 8704 and pe.mx_bytes(129, 128) == 2 * 8704
    assert pe.mx_bytes(14, 2880) == 23 * 8704 and pe.mx_bytes(201088, 2880) == 1571 * 23 * 8704
    assert pe.mx_bytes(1 << 24, 1 << 20) == 8704 << 30  # beyond 32 bits
    assert pe.mx_bytes(0, 5) == 0 and pe.mx_bytes(-1, 5) == 0 and pe.mx_bytes(5, 0) == 0
    assert pe.mx_bytes((1 << 24) + 1, 5) == 0 and pe.mx_bytes(5, (1 << 20) + 1) == 0
    for n, w in ((14, 2880), (1, 1), (300, 129)):
        assert int(pe.lib().pe_linear_mx_workspace_bytes(n, w)) >= pe.mx_bytes(n, w)
    assert int(pe.lib().pe_linear_mx_workspace_bytes(-1, 3)) == 0


# ----------------------------------------------------------------------------- refusals

def _rows(call, dtype=1, x=AT, stride=256, n=0, width=256, mat=1 << 50, err=1 << 51):
    if call == "q":
        return pe.lib().pe_quantize_mx(dtype, _p(x), stride, n, width, _p(mat), _p(err), NULL)
    return pe.lib().pe_dequantize_mx(dtype, _p(mat), n, width, _p(x), stride, NULL)


@pytest.mark.parametrize("call", ["q", "d"])
def test_quantise_and_read_back_refuse_before_launch(call):
    assert _rows(call) == 0 and _rows(call, stride=257) == 0 and _rows(call, x=AT + 2) == 0  # no rows: fine
    assert _rows(call, dtype=2) == 1 and _rows(call, dtype=-1) == 1
    assert _rows(call, x=None) == 1 and _rows(call, mat=None) == 1
    assert _rows(call, x=AT + 1) == 1 and _rows(call, dtype=0, x=AT + 2) == 1  # between elements
    assert _rows(call, mat=(1 << 50) + 8) == 1
    assert _rows(call, stride=255) == 1
    assert _rows(call, n=-1) == 2 and _rows(call, n=(1 << 24) + 1) == 2
    assert _rows(call, width=0) == 2 and _rows(call, width=(1 << 20) + 1, stride=1 << 21) == 2
    assert _rows(call, n=4, mat=AT + 512) == 1       # the matrix inside the rows
    assert _rows(call, n=4, mat=AT - 16 * 512) == 1  # and the rows inside the matrix
    if call == "q":
        assert _rows(call, err=None) == 1


def _matmul(x=1 << 50, n=0, w=1 << 51, m=512, width=256, add=None, add_stride=512, dtype=1, y=AT, ys=512, err=1 << 52):
    return pe.lib().pe_matmul_mx(_p(x), n, _p(w), m, width, _p(add), add_stride, dtype, _p(y), ys, _p(err), NULL)


def _linear(x=1 << 50, n=0, w=1 << 51, m=512, width=256, add=None, add_stride=512, dtype=1, y=AT, ys=512, err=1 << 52,
            xd=1, xs=256, ws=1 << 53, wsb=1 << 30):
    return pe.lib().pe_linear_mx(xd, _p(x), xs, n, _p(w), m, width, _p(add), add_stride, dtype, _p(y), ys, _p(ws), wsb,
                                 _p(err), NULL)


@pytest.mark.parametrize("call", [_matmul, _linear])
def test_products_refuse_before_launch(call):
    assert call() == 0 and call(add=AT) == 0 and call(add=1 << 54) == 0 and call(ys=517, y=AT + 2) == 0
    for name in ("x", "w", "y", "err"):
        assert call(**{name: None}) == 1, name
    assert call(w=(1 << 51) + 8) == 1 and call(y=AT + 1) == 1 and call(dtype=0, y=AT + 2) == 1
    assert call(dtype=7) == 1 and call(ys=511) == 1 and call(add=1 << 54, add_stride=511) == 1
    assert call(n=-1) == 2 and call(m=0) == 2 and call(m=(1 << 24) + 1, ys=1 << 25) == 2 and call(width=0, xs=256) == 2 \
        if call is _linear else call(n=-1) == 2 and call(m=0) == 2 and call(width=0) == 2
    # y among the weights, among x, or over another part of add
    assert call(n=4, w=AT) == 1 and call(n=4, w=AT - 8704 * 4) == 1
    assert call(n=4, x=AT) == 1
    assert call(n=4, add=AT + 16) == 1 and call(n=4, add=AT, add_stride=520) == 1


def test_linear_refuses_workspaces():
    assert _linear(ws=None) == 1 and _linear(ws=(1 << 53) + 128) == 1
    need = int(pe.lib().pe_linear_mx_workspace_bytes(4, 256))
    assert _linear(n=4, wsb=need - 1) == 2
    for name in ("x", "y", "w", "add"):
        assert _linear(n=4, **{name: 1 << 53}) == 1, name
    assert _linear(x=AT + 1) == 1 and _linear(xs=255) == 1 and _linear(xd=3) == 1
    # y beside x in one buffer, with one stride, is apart; over it, it is not
    assert _linear(n=4, x=AT, xs=1024, y=AT + 2 * 255, ys=1024) == 1


def test_matmul_refuses_misaligned_x():
    assert _matmul(x=(1 << 50) + 8) == 1


def _cfg(**kw):
    base = dict(B=3, K=1, d=64, n_q=8, n_kv=2, head_dim=64, ffn=64, vocab=2, n_layers=1, max_pages_per_seq=9,
                dtype="bf16")
    base.update(kw)
    return pe.Config.make(**base)


def _append(cfg, q=1 << 50, k=1 << 51, v=1 << 52, qs=512, ks=128, vs=128, pos=1 << 53, axes=1, of=None, slots=1 << 54,
            n=0, qo=1 << 55, qos=512, kc=1 << 56, vc=1 << 57, pages=4, err=1 << 58):
    return pe.lib().pe_append_kv(ctypes.byref(cfg), _p(q), _p(k), _p(v), qs, ks, vs, _p(pos), axes, of, _p(slots), n,
                                 _p(qo), qos, _p(kc), _p(vc), pages, _p(err), NULL)


def _append_packed(cfg, q=1 << 50, k=1 << 51, v=1 << 52, qs=512, ks=128, vs=128, pos=1 << 53, axes=1, of=None,
                   slots=1 << 54, n=0, qo=1 << 55, qos=512, kc=1 << 56, pages=4, err=1 << 58):
    return pe.lib().pe_append_kv_packed(ctypes.byref(cfg), _p(q), _p(k), _p(v), qs, ks, vs, _p(pos), axes, of, _p(slots),
                                        n, _p(qo), qos, _p(kc), pages, _p(err), NULL)


@pytest.mark.parametrize("call", [_append, _append_packed])
def test_append_refuses_before_launch(call):
    c = _cfg()
    assert call(c) == 0 and call(c, q=None, qo=None) == 0 and call(c, qo=1 << 50) == 0
    for name in ("k", "v", "pos", "slots", "kc", "err"):
        assert call(c, **{name: None}) == 1, name
    assert call(c, q=None) == 1 and call(c, qo=None) == 1
    for name in ("q", "k", "v", "qo", "kc"):
        assert call(c, **{name: AT + 8}) == 1, name
    for name, width in (("qs", 512), ("ks", 128), ("vs", 128), ("qos", 512)):
        assert call(c, **{name: width - 1}) == 1 and call(c, **{name: width + 4}) == 1, name
    assert call(c, n=-1) == 2 and call(c, pages=0) == 2 and call(c, axes=0) == 2 and call(c, axes=9) == 2
    assert call(c, axes=3, of=bytes([0, 1, 2, 2] * 8)) == 0 and call(c, axes=2, of=bytes([0, 1, 2, 2] * 8)) == 1
    for bad, status in ((dict(head_dim=96), 3), (dict(n_q=7), 2), (dict(n_kv=0), 2), (dict(rope_theta=0.0), 1),
                        (dict(rope_theta=float("inf")), 1), (dict(rope_theta=float("nan")), 1)):
        assert call(_cfg(**bad)) == status, bad
    # outputs over inputs: q_out over k, over q with another stride; the cache over rows
    assert call(c, n=4, qo=1 << 51) == 1 and call(c, n=4, qo=1 << 50, qos=520) == 1
    assert call(c, n=4, kc=1 << 51) == 1 and call(c, n=4, kc=1 << 55) == 1


def test_append_refuses_caches_that_overlap():
    c = _cfg()
    assert _append(c, n=4, vc=1 << 56) == 1 and _append(c, n=4, vc=(1 << 56) + 16) == 1
    assert _append(c, n=4, vc=1 << 50) == 1 and _append(c, n=4, vc=1 << 52) == 1


@pytest.mark.parametrize("name", ["pe_draft_forward_mx_head", "pe_step_mx_head"])
def test_drafter_calls_with_a_4_bit_head_refuse_before_launch(name):
    c = _cfg(d=128, ffn=128, vocab=300)
    layer = (ctypes.c_void_p * 1)(1 << 49)
    w = pe._Weights(AT, AT, AT, layer, layer, layer, layer, layer, layer, AT, None)
    kv, packed = pe._KV(layer, layer, 40), pe._PackedKV(layer, 40)
    need = pe.lib().pe_mx_head_workspace_bytes(ctypes.byref(c))
    assert need >= pe.packed_workspace_bytes(c) + pe.mx_bytes(c.B * c.K, c.d)
    assert pe.lib().pe_mx_head_workspace_bytes(ctypes.byref(_cfg(d=100))) == 0

    def call(head=1 << 52, kv=ctypes.byref(kv), packed=None, ws=1 << 47, wsb=need, drop=None, weights=w):
        ptrs = [_p((1 << 40) + i * (1 << 32)) for i in range(7)]
        outs = [_p((1 << 40) + (20 + i) * (1 << 32)) for i in range(3 if "forward" in name else 7)]
        if drop is not None:
            ptrs[drop] = None
        return getattr(pe.lib(), name)(ctypes.byref(c), ctypes.byref(weights), _p(head), kv, packed, *ptrs, _p(ws),
                                       ctypes.c_size_t(wsb), *outs, NULL)

    assert call(wsb=need - 1) == 2 and call(wsb=pe.packed_workspace_bytes(c)) == 2
    assert call(kv=None, packed=ctypes.byref(packed), wsb=need - 1) == 2
    assert call(head=None) == 1 and call(head=(1 << 52) + 8) == 1 and call(ws=(1 << 47) + 128) == 1
    assert call(kv=None) == 1 and call(packed=ctypes.byref(packed)) == 1
    for i in range(7):
        assert call(drop=i) == 1
    assert call(weights=pe._Weights(AT, AT, None, layer, layer, layer, layer, layer, layer, AT, None)) == 1


def test_the_binding_refuses_what_is_no_gpu_tensor_or_no_matrix():
    m, err = pe.MxMatrix(2, 32, device="cpu"), torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(2, 32)
    calls = [lambda: pe.quantize_mx(x, m, err), lambda: pe.dequantize_mx(m, x), lambda: pe.matmul_mx(m, m, x, err),
             lambda: pe.linear_mx(x, m, x, m.data, err), lambda: pe.quantize_mx(None, m, err),
             lambda: pe.linear_mx([1.0], m, 3, m.data, err),
             lambda: pe.append_kv(_cfg(), x, x, x, err, torch.zeros(2, dtype=torch.int64), (x, x), x, err),
             lambda: pe.append_kv(_cfg(), x, x, x, err, None, (x, x), x, err)]
    for call in calls:
        with pytest.raises(ValueError):
            call()
    with pytest.raises((TypeError, ValueError)):
        pe.append_kv(b"12", x, x, x, err, torch.zeros(2, dtype=torch.int64), (x, x), x, err)
