"""Long sums of attend_packed in fp32: tensor cores cut what they add to an accumulator instead of rounding it, so a sum that
ran through one accumulator would fall short by an amount that grows with its length.

The bound on the mean of (output - formula) / formula, all values positive, holds whatever the length:
  2^-20        the exponent's error, as in test_gpu_packed.py;
  3 * 2^-23    a page's sum: three products, each cut by less than a step;
  2 * hd/16 * 3 * 2^-23 * depth   scores, sums of hd/16 * 3 products, at most `depth` (queries are small here), acting on
               the weights and on their sum.
Every page's sum is then added with fp32's rounding, whose errors have no sign: their mean over these 131,072 outputs or
more, sqrt(L/16) * 2^-24 / sqrt(131072) at most for errors of one size, is below 2^-27.
"""

import pytest
import torch

import speculative_decoding_step_gb300 as pe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [1, 4])
@pytest.mark.parametrize("L", [1000, 16384])
def test_attend_f32_long_sums_do_not_fall_short(L, rows, hd):
    B, n_q, n_kv = 64, 32, 8
    pages = -(-L // 16)
    cfg = pe.Config.make(B, 1, 64, n_q, n_kv, hd, 64, 2, 1, pages, "f32")
    g = torch.Generator(device="cuda").manual_seed(L + rows + hd)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    pool, err = pe.alloc_packed_pool(cfg, pages), torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.arange(L, device="cuda")
    pe.pack_kv(cfg, rnd(L, n_kv, hd), (1 + rnd(L, n_kv, hd).abs()) * (1 + torch.rand(hd, device="cuda", generator=g)), slots,
               pool, err)
    k, v = (torch.empty((L, n_kv, hd), device="cuda") for _ in range(2))
    pe.unpack_kv(cfg, pool, slots, k, v, err)
    n = B * rows
    q, out = rnd(n, n_q * hd) / 64, torch.empty((n, n_q * hd), device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B, 1)  # one cache for every sequence
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda") * rows
    pe.attend_packed(cfg, q, pool, table, start, torch.full((n,), L - 1, dtype=torch.int32, device="cuda"), rows, out,
                     pe.alloc_attend_workspace(cfg), err)
    assert int(err.item()) == 0
    off, depth = [], 0.0
    for h in range(n_kv):
        x = q.double().view(n, n_kv, -1, hd)[:, h].flatten(0, 1)
        w = torch.softmax(x @ k[:, h].double().T / hd ** 0.5, -1)
        want = (w @ v[:, h].double()).view(n, -1, hd)
        depth = max(depth, float((x.abs() @ k[:, h].double().abs().T).max()) / hd ** 0.5)
        off.append(out.double().view(n, n_kv, -1, hd)[:, h] / want - 1)
    bound = 2.0 ** -20 + 3 * 2.0 ** -23 + 2 * (hd // 16) * 3 * 2.0 ** -23 * depth
    assert abs(float(torch.stack(off).mean())) <= bound, (float(torch.stack(off).mean()), bound, depth)
