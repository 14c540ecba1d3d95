"""The packed (4-bit) KV cache and the attention over it, in 64 bits, from the format's definition.

Blocks of 16 consecutive entries of a head's row share the scale byte c, s(c) = (1 + (c & 7)/8) *
2^((c >> 3) - 19), the smallest with 7 s(c) >= the block's largest finite magnitude; entry x is
kept as n = sign(x) min(7, floor(|x|/s + 1/2)) and stands for n s.  A page's record per kv head is
key codes, value codes, key scales, value scales (rows by position); a code row is 32-bit words
of eight nibbles n + 8.
"""

from __future__ import annotations

import numpy as np

PAGE, BLOCK = 16, 16
SCALES = np.array([(1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 19) for c in range(256)])


def quantise(x: np.ndarray):
    """Rows x [..., hd] -> (n [..., hd] int, scale bytes [..., hd/16])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    finite = np.isfinite(b)
    amax = np.where(finite, np.abs(b), 0).max(-1)
    byte = np.minimum(np.searchsorted(7 * SCALES, amax, side="left"), 255)
    s = SCALES[byte][..., None]
    with np.errstate(invalid="ignore"):
        n = np.sign(b) * np.minimum(7, np.floor(np.abs(b) / s + 0.5))
    n = np.where(np.isnan(b), 0, n)
    return n.reshape(x.shape).astype(np.int64), byte.astype(np.uint8)


def kept(x: np.ndarray) -> np.ndarray:
    """What the packed form keeps of rows x."""
    n, byte = quantise(x)
    return n * np.repeat(SCALES[byte], BLOCK, axis=-1)


def nibble_of(hd: int, values: bool) -> np.ndarray:
    """Index of each entry's nibble in its row."""
    at = np.empty(hd, dtype=np.int64)
    for e in range(hd):
        block, r = divmod(e, BLOCK)
        if values:
            half, j = divmod(block, 4)
            at[e] = 8 * ((r % 8) * (hd // 64) + half) + 2 * j + r // 8
        else:
            t, odd = divmod(r, 4)
            at[e] = 8 * (t * (hd // 32) + block // 2) + 2 * (block % 2) + odd // 2 + 4 * (odd % 2)
    return at


def code_row(n: np.ndarray, values: bool) -> np.ndarray:
    """n [..., hd] -> bytes [..., hd/2]."""
    hd = n.shape[-1]
    nib = np.empty_like(n)
    nib[..., nibble_of(hd, values)] = n + 8
    return (nib[..., 0::2] | nib[..., 1::2] << 4).astype(np.uint8)


def write(pool: np.ndarray, k: np.ndarray, v: np.ndarray, slots: np.ndarray) -> None:
    """Packs rows k, v [n][n_kv][hd] into pool [pages][n_kv][18*hd] at slots (negative: passed over)."""
    hd = k.shape[-1]
    for base, x, values in ((0, k, False), (8 * hd, v, True)):
        n, byte = quantise(x)
        rows = code_row(n, values)
        sbase = 17 * hd if values else 16 * hd
        for i, slot in enumerate(slots):
            if slot < 0:
                continue
            page, off = divmod(int(slot), PAGE)
            pool[page, :, base + off * (hd // 2): base + (off + 1) * (hd // 2)] = rows[i]
            pool[page, :, sbase + off * (hd // 16): sbase + (off + 1) * (hd // 16)] = byte[i]


def read(pool: np.ndarray, slots: np.ndarray):
    """Entries at slots as the values they stand for: (k, v) [n][n_kv][hd]."""
    hd = pool.shape[-1] // 18
    page, off = np.asarray(slots) // PAGE, np.asarray(slots) % PAGE
    out = []
    for base, sbase, values in ((0, 16 * hd, False), (8 * hd, 17 * hd, True)):
        codes = pool[..., base:base + 8 * hd].reshape(*pool.shape[:2], PAGE, hd // 2)[page, :, off]
        scale = pool[..., sbase:sbase + hd].reshape(*pool.shape[:2], PAGE, hd // 16)[page, :, off]
        nib = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], hd).astype(np.int64)
        n = nib[..., nibble_of(hd, values)] - 8
        out.append(n * np.repeat(SCALES[scale], BLOCK, axis=-1))
    return out


def attend(q, pool, block_table, row_start, positions, n_q):
    """(out, size, depth) of rows q [n][n_q*hd]: the attention; the same sum over |values| (what errors of
    the weights scale with); the largest sum over |q_e k_e| / sqrt(hd) that a row's scores are made of.
    A page outside the pool counts as zero keys and values; a position -1 gives zeros."""
    n_kv, hd = pool.shape[1], pool.shape[-1] // 18
    G, n = n_q // n_kv, len(positions)
    qd = np.asarray(q, dtype=np.float64).reshape(n, n_kv, G, hd)
    out, size, depth = np.zeros_like(qd), np.zeros_like(qd), np.zeros((n, n_q))
    for b in range(len(row_start) - 1):
        for r in range(row_start[b], row_start[b + 1]):
            L = int(positions[r]) + 1
            if L <= 0:
                continue
            x = np.arange(L)
            page = block_table[b, x // PAGE].astype(np.int64)
            good = (page >= 0) & (page < pool.shape[0])
            k, v = read(pool, np.where(good, page, 0) * PAGE + x % PAGE)
            k, v = k * good[:, None, None], v * good[:, None, None]
            s = np.einsum("ngd,lnd->ngl", qd[r], k) / np.sqrt(hd)
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out[r] = np.einsum("ngl,lnd->ngd", w, v)
            size[r] = np.einsum("ngl,lnd->ngd", w, np.abs(v))
            depth[r] = (np.einsum("ngd,lnd->ngl", np.abs(qd[r]), np.abs(k)).max(-1) / np.sqrt(hd)).reshape(-1)
    return out.reshape(n, -1), size.reshape(n, -1), np.repeat(depth, hd, axis=1)


def entry_bytes(shape, slots) -> np.ndarray:
    """Mask over a pool of this shape: the bytes that hold the entries at slots."""
    hd = shape[-1] // 18
    mask = np.zeros(shape, dtype=bool)
    for slot in slots:
        page, off = divmod(int(slot), PAGE)
        for base, row in ((0, hd // 2), (8 * hd, hd // 2), (16 * hd, hd // 16), (17 * hd, hd // 16)):
            mask[page, :, base + off * row: base + (off + 1) * row] = True
    return mask


def draft_forward(cfg, weights, x0_rows, positions, seqs, block_table, pools, draft_rows) -> dict:
    """The drafter pass over packed caches that hold the pass's own rows already (as the pass left them).

    The pass of ``oracle.draft_forward`` with every key and value taken from ``pools`` (one per layer), so that
    the result depends on its inputs without the jumps of rounding to 4 bits.  Rows are in sequence order.
    Returns logits [n_draft][V] and, per layer, the k (post-RoPE) and v [n][n_kv][hd] of the rows before they are
    packed."""
    from . import linear, rmsnorm, rope, widen
    hd, nq, nkv = cfg.head_dim, cfg.n_q, cfg.n_kv
    x0 = np.asarray(x0_rows)
    n = len(positions)
    row_start = np.searchsorted(np.asarray(seqs), np.arange(len(block_table) + 1))
    X = linear(x0 if x0.dtype == np.float64 else widen(x0), weights.fc)
    ks, vs = [], []
    for l in range(cfg.n_layers):
        h = linear(rmsnorm(X, weights.norm_attn[l], cfg.rms_eps), weights.wqkv[l]).reshape(n, nq + 2 * nkv, hd)
        for i in range(n):
            for g in range(nq + nkv):
                h[i, g] = rope(h[i, g], positions[i], cfg.rope_theta)
        ks.append(h[:, nq:nq + nkv])
        vs.append(h[:, nq + nkv:])
        out, _, _ = attend(h[:, :nq].reshape(n, -1), pools[l], block_table, row_start, positions, nq)
        X = X + linear(out, weights.wo[l])
        gu = linear(rmsnorm(X, weights.norm_mlp[l], cfg.rms_eps), weights.w_gate_up[l])
        gate, up = gu[:, :cfg.ffn], gu[:, cfg.ffn:]
        X = X + linear(gate / (1 + np.exp(-gate)) * up, weights.w_down[l])
    last = rmsnorm(X[np.asarray(draft_rows)], weights.norm_final, cfg.rms_eps)
    return dict(logits=linear(last, weights.lm_head), new_k=ks, new_v=vs)
