"""Measured cases of the microscaled 4-bit matrices and of appending rotated rows to a KV cache.

Five operators of the package are measured here, each through its public call:

* ``quantize_mx``    rows rounded to 4-bit floating point with a power-of-two scale per 32 entries;
* ``dequantize_mx``  such a matrix read back as the values it stands for;
* ``matmul_mx``      the product of two such matrices, optionally added to rows that are there;
* ``linear_mx``      the same from rows in full precision, which are quantised on the way;
* ``append_kv``      query and key rows rotated by their positions (of one or several axes), keys and
  values written into a paged cache.

A block of 32 consecutive entries of a row shares the scale 2^e, e = floor(log2 of the block's
largest magnitude) - 2, between -127 and 127 (-127 for a block of zeros).  An entry x is kept as the
nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 to |x| 2^-e (of two equally near ones the one whose code, its
place in that list, is even; 6 beyond 6), with x's sign.
"""

import math

import torch

own = False

PAGE = 16
BLOCK = 32
THETA = 10000.0
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------- the cases

def listed():
    # Widths, feature counts and heads of the drafters that the benchmark runs (width 2880, 64 query heads
    # over 8 of 64 dims, 7680 hidden features, 201088 tokens; width 2048, 32 heads over 4 of 128, 6144
    # hidden features) and of its small fp32 configuration (width 256, 4 heads over 4 of 64).
    bf, f32 = dict(dtype="bf16"), dict(dtype="f32")
    return [
        # one user's draft rows before a projection: latency is all there is
        dict(name="quantize-draft-B1", op="quantize", rows=14, width=2880, pad=0, mix=1, **bf),
        # the hidden features of a batch of prompts
        dict(name="quantize-prompts", op="quantize", rows=8209, width=7680, pad=0, mix=2, **bf),
        # a gate-and-up matrix read back, as a program does that folds another matrix into it
        dict(name="read-gate-up", op="read", rows=15360, width=2880, pad=0, mix=3, **bf),
        # a small matrix of odd width, rows apart
        dict(name="read-odd-f32", op="read", rows=131, width=257, pad=7, mix=4, **f32),
        # a full batch's draft rows, quantised once for several matrices: the query, key and value heads
        dict(name="matmul-qkv-B64", op="matmul", rows=640, width=2880, n_out=5120, add=False, out="bf16", pad=0, mix=5, **bf),
        # a long prompt's rows through gate and up
        dict(name="matmul-gate-up-prompt", op="matmul", rows=4099, width=2048, n_out=12288, add=False, out="bf16", pad=0, mix=6, **bf),
        # the small configuration's heads
        dict(name="linear-small-f32", op="linear", rows=8, width=256, n_out=768, add=False, out="f32", pad=0, mix=7, **f32),
        # one user's draft rows through gate and up
        dict(name="linear-gate-up-B1", op="linear", rows=14, width=2880, n_out=15360, add=False, out="bf16", pad=0, mix=8, **bf),
        # a full batch's rows back to the residual stream
        dict(name="linear-down-B64", op="linear", rows=896, width=7680, n_out=2880, add=True, out="f32", pad=0, mix=9, **bf),
        # one user's draft rows to logits over the whole vocabulary
        dict(name="linear-logits-B1", op="linear", rows=7, width=2880, n_out=201088, add=False, out="f32", pad=0, mix=10, **bf),
        # one new token for each of 64 users
        dict(name="append-token-B64", op="append", rows=64, n_q=64, n_kv=8, hd=64, axes=1, mix=11, **bf),
        # two prompts with pictures: time, height and width; some rows go to no slot
        dict(name="append-prompts", op="append", rows=8198, n_q=32, n_kv=4, hd=128, axes=3, mix=12, **bf),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["quantize", "read", "matmul", "linear", "linear", "append"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    mix = rng.randrange(1 << 30)
    if op == "append":
        n_kv, hd = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        return dict(op=op, rows=_spread(rng, 1, 8192), n_q=n_kv * rng.choice([1, 2, 4, 5, 8]), n_kv=n_kv, hd=hd,
                    axes=rng.choice([1, 1, 2, 3]), dtype=dtype, mix=mix)
    width = _spread(rng, 32, 8192)
    if rng.random() < 0.6:                       # widths of whole blocks, as models have them
        width = -(-width // 32) * 32
    pad = rng.choice([0, 0, 8, 24, 3])
    if op in ("quantize", "read"):
        return dict(op=op, rows=_spread(rng, 1, 8192), width=width, pad=pad, dtype=dtype, mix=mix)
    n_out = _spread(rng, 1, 32768)
    n_out = min(n_out, (1 << 26) // width)
    rows = _spread(rng, 1, 4096)
    rows = max(1, min(rows, (1 << 35) // (width * n_out)))
    return dict(op=op, rows=rows, width=width, n_out=n_out, add=rng.random() < 0.4, out=rng.choice(["bf16", "f32"]),
                pad=pad, dtype=dtype, mix=mix)


def _bytes(dtype):
    return 2 if dtype == "bf16" else 4


def work(case):
    n, eb = case["rows"], _bytes(case["dtype"])
    if case["op"] == "append":
        row = (case["n_q"] + 2 * case["n_kv"]) * case["hd"] * eb
        return dict(bytes=2 * n * row + (8 + 4 * case["axes"]) * n, flops=3 * n * (case["n_q"] + case["n_kv"]) * case["hd"])
    k = case["width"]
    held = -(-k // BLOCK) * 17                   # bytes of a row in 4 bits: 16 of codes and a scale per block
    if case["op"] == "quantize":                 # quantised, and what was kept is read back
        return dict(bytes=2 * n * (k * eb + held), flops=0)
    if case["op"] == "read":
        return dict(bytes=n * (k * eb + held), flops=0)
    m, ob = case["n_out"], _bytes(case["out"])
    x = n * held if case["op"] == "matmul" else n * k * eb
    return dict(bytes=x + m * held + n * m * ob * (2 if case["add"] else 1), flops=2 * n * m * k)


# ----------------------------------------------------------------------------- inputs

def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _source(case, seed):
    """The inputs themselves: rows, weights, what is added; for appending the rows, positions, slots and cache."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + case["mix"] % 1000003)
    rnd = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    n, dt = case["rows"], _dt(case["dtype"])
    if case["op"] == "append":
        n_q, n_kv, hd = case["n_q"], case["n_kv"], case["hd"]
        size = torch.exp(0.4 * rnd(n_q + 2 * n_kv, hd))          # channels differ in size
        # as a fused projection leaves them: queries, keys and values side by side
        qkv = (rnd(n, n_q + 2 * n_kv, hd) * size).to(dt)
        # time goes on from a cached context; height and width are those of pictures on the way
        first = int(torch.randint(1, 100000, (1,), device="cuda", generator=g))
        time = first + torch.arange(n, device="cuda")
        pos = [time, first + (time // 37) % 64, first + time % 37][: case["axes"]]
        pages = n // PAGE + 8
        slots = torch.randperm(pages * PAGE, device="cuda", generator=g)[:n]
        if n > 100:
            slots[5::23] = -1
        axis = [(i * case["axes"]) // (hd // 2) for i in range(hd // 2)]
        cache = rnd(2, pages, PAGE, n_kv, hd).to(dt)
        return dict(qkv=qkv, positions=torch.stack(pos).int(), slots=slots, axis=axis, cache=cache)
    k = case["width"]
    s = {}
    room = rnd(n, k + case["pad"])
    room *= torch.exp(0.5 * rnd(k + case["pad"]))                # channels differ in size, a few by much
    if case["op"] == "read":
        room *= 0.02
    s["x"] = room.to(dt)[:, :k]
    if "n_out" in case:
        m = case["n_out"]
        s["w"] = rnd(m, k).mul_(0.02).to(torch.bfloat16)
        if case["add"]:
            s["add"] = rnd(n, m).to(_dt(case["out"]))
    return s


def prepare(case, seed):
    src = _source(case, seed)
    st = dict(case=case)
    dev = dict(device="cuda")
    n = case["rows"]
    if own:
        import speculative_decoding_step_gb300 as pe
        st["pe"], st["err"] = pe, torch.zeros(1, dtype=torch.int32, **dev)
    if case["op"] == "append":
        n_q, n_kv, hd = case["n_q"], case["n_kv"], case["hd"]
        st.update(q=src["qkv"][:, :n_q], k=src["qkv"][:, n_q:n_q + n_kv], v=src["qkv"][:, n_q + n_kv:],
                  positions=src["positions"], slots=src["slots"], k_cache=src["cache"][0].clone(),
                  v_cache=src["cache"][1].clone(), q_out=torch.empty((n, n_q * hd), dtype=src["qkv"].dtype, **dev))
        st["axis"] = torch.tensor(src["axis"], **dev)
        st["freq"] = THETA ** (-2.0 * torch.arange(hd // 2, dtype=torch.float64, **dev) / hd)
        if own:
            st["cfg"] = pe.Config.make(1, 1, 64, n_q, n_kv, hd, 64, 2, 1, 1, case["dtype"], rope_theta=THETA)
            st["axes"] = bytes(src["axis"])
        return st
    k = case["width"]
    if case["op"] == "linear" or case["op"] == "quantize":
        st["x"] = src["x"]
    if case["op"] in ("quantize", "read"):
        st["out"] = torch.empty((n, k + case["pad"]), dtype=_dt(case["dtype"]), **dev)[:, :k]
    if "n_out" in case:
        st["y"] = torch.empty((n, case["n_out"]), dtype=_dt(case["out"]), **dev)
        st["add"] = src.get("add")
    st["levels"] = torch.tensor(LEVELS + tuple(-v for v in LEVELS), **dev)
    st["powers"] = torch.tensor([2.0 ** (i - 127) for i in range(255)], **dev)
    # the matrices that are there in 4 bits before the call
    for name, needed in (("xq", case["op"] in ("read", "matmul")), ("wq", "n_out" in case)):
        if not needed:
            continue
        rows = src["x" if name == "xq" else "w"]
        if own:
            st[name] = pe.MxMatrix(rows.shape[0], k)
            pe.quantize_mx(rows, st[name], st["err"])
        else:
            st[name] = _in_pieces(rows)
    if own and case["op"] == "quantize":
        st["xq"] = pe.MxMatrix(n, k)
    if own and case["op"] == "linear":
        st["workspace"] = pe.alloc_linear_mx_workspace(n, k)
    return st


def _in_pieces(rows):
    """Plain codes and scales of many rows, made some 100 MB at a time."""
    step = max(1, (1 << 24) // rows.shape[1])
    parts = [_quantise(rows[a:a + step]) for a in range(0, rows.shape[0], step)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


# ----------------------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if op == "append":
        if own:
            st["pe"].append_kv(st["cfg"], st["q"], st["k"], st["v"], st["positions"], st["slots"],
                               (st["k_cache"], st["v_cache"]), st["q_out"], st["err"], axes=st["axes"])
        else:
            _plain_append(st)
        return dict(q=st["q_out"], k_cache=st["k_cache"], v_cache=st["v_cache"])
    if own:
        pe, err = st["pe"], st["err"]
        if op == "quantize":
            pe.quantize_mx(st["x"], st["xq"], err)
        if op in ("quantize", "read"):
            pe.dequantize_mx(st["xq"], st["out"])
        elif op == "matmul":
            pe.matmul_mx(st["xq"], st["wq"], st["y"], err, add=st["add"])
        else:
            pe.linear_mx(st["x"], st["wq"], st["y"], st["workspace"], err, add=st["add"])
    elif op in ("quantize", "read"):
        held = _quantise(st["x"]) if op == "quantize" else st["xq"]
        st["out"].copy_(_values(held, st)[:, : case["width"]])
    else:
        xq = st["xq"] if op == "matmul" else _quantise(st["x"])
        y = _values(xq, st) @ _values(st["wq"], st).t()
        if st["add"] is not None:
            y = y + st["add"].float()
        st["y"].copy_(y)
    return dict(out=st["out"] if op in ("quantize", "read") else st["y"])


def _quantise(x):
    """Code bytes (two entries each, the first in the lower half) and scale exponents + 127 of rows x."""
    short = -x.shape[1] % BLOCK
    b = torch.nn.functional.pad(x.float(), (0, short)).unflatten(1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top)[1] - 3).clamp_(-127, 127)
    e = torch.where(top == 0, -127, e)
    a = torch.ldexp(b.abs().double(), -e)
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code | (torch.signbit(b).to(torch.uint8) << 3)).flatten(1)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _values(held, st):
    """The fp32 values that codes and scales stand for, with the entries that fill up the last block."""
    codes, scales = held
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(1)
    return (st["levels"][code.int()].unflatten(1, (-1, BLOCK)) * st["powers"][scales.int()].unsqueeze(-1)).flatten(1)


def _plain_append(st):
    turn = st["positions"].double()[st["axis"]].t() * st["freq"]     # [n][hd/2], angles in 64 bits
    c, s = torch.cos(turn).float().unsqueeze(1), torch.sin(turn).float().unsqueeze(1)

    def rotated(x):
        a, b = x.float().chunk(2, -1)
        return torch.cat((a * c - b * s, b * c + a * s), -1).to(x.dtype)

    st["q_out"].copy_(rotated(st["q"]).flatten(1))
    keep = st["slots"] >= 0
    at = st["slots"][keep]
    st["k_cache"].flatten(0, 1)[at] = rotated(st["k"])[keep]
    st["v_cache"].flatten(0, 1)[at] = st["v"][keep]


# ----------------------------------------------------------------------------- in 64 bits

def _kept(x):
    """What the 4-bit form keeps of rows x, from the definition: no codes are made."""
    x = x.double()
    short = -x.shape[1] % BLOCK
    b = torch.cat((x, x.new_zeros(x.shape[0], short)), 1).view(x.shape[0], -1, BLOCK)
    top = b.abs().max(-1, keepdim=True).values
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -200)))
    e = torch.where(torch.exp2(e) > top, e - 1, e)                   # log2 rounds; the powers do not
    e = torch.where(torch.exp2(e + 1) <= top, e + 1, e)
    unit = torch.exp2((e - 2).clamp(-127, 127))
    a = b.abs() / unit
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6)                  # halves to the even neighbour
    return (torch.sign(b) * a * unit).view(x.shape[0], -1)[:, : x.shape[1]]


def exact(case, seed):
    src = _source(case, seed)
    if case["op"] == "append":
        n_q, n_kv, hd, n = case["n_q"], case["n_kv"], case["hd"], case["rows"]
        x = src["qkv"].double()
        out = x.clone()
        for i in range(hd // 2):
            angle = src["positions"][src["axis"][i]].double() * math.pow(THETA, -2.0 * i / hd)
            c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
            a, b = x[:, : n_q + n_kv, i], x[:, : n_q + n_kv, i + hd // 2]
            out[:, : n_q + n_kv, i] = a * c - b * s
            out[:, : n_q + n_kv, i + hd // 2] = a * s + b * c
        cache = src["cache"].double().flatten(1, 2)
        put = (src["slots"] >= 0).nonzero().squeeze(1)
        cache[0, src["slots"][put]] = out[put, n_q:n_q + n_kv]
        cache[1, src["slots"][put]] = out[put, n_q + n_kv:]
        cache = cache.view(src["cache"].shape)
        return dict(q=out[:, :n_q].reshape(n, n_q * hd), k_cache=cache[0], v_cache=cache[1])
    kept = _kept(src["x"])
    if "n_out" not in case:
        return dict(out=kept)
    step = max(1, (1 << 27) // case["width"])                        # weights, a GB of 64 bits at a time
    y = torch.cat([kept @ _kept(src["w"][a:a + step]).t() for a in range(0, case["n_out"], step)], 1)
    return dict(out=y + src["add"].double() if case["add"] else y)
