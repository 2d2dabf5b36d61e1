"""The operators on matrices in microscaled 4-bit floating point, as they are measured: quantising
(and reading back), the product of two such matrices, and a linear layer's passes over them.

A matrix is held as 4-bit codes (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) with one power of two
for each 32 consecutive columns of a row. Codes: uint8 [rows][16 * ceil(cols / 32)], the lower four
bits the even column. Exponents (biased by 127): tiles of 128 rows by 4 blocks, 512 bytes each, in
which row r and block b lie at (r % 32) * 16 + (r / 32) * 4 + b.

``run`` computes them in elementary torch operations, or, where ``own`` is true, makes the calls
a user makes of the library.
"""
import math

import torch

own = False

BLOCK = 32
GOLDEN, MIX_A, MIX_B, MIX_C = 0x9E3779B9, 0x9016D2F5, 0x314549A1, 0x8A8866C7
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------------------------
# the cases

def listed():
    return [
        # a small layer's weights after a step, odd sizes: latency of one call
        {"name": "quantize small", "op": "quantize", "rows": 197, "cols": 1000, "in": "f32",
         "forms": "rows", "rounding": "nearest", "residual": False, "pad": 0},
        # an embedding's fp32 master weights after a step, for the forward and the backward product
        {"name": "quantize embedding", "op": "quantize", "rows": 30522, "cols": 1024, "in": "f32",
         "forms": "both", "rounding": "nearest", "residual": False, "pad": 0},
        # gradients of 8192 tokens, unbiased, for both products of the backward pass
        {"name": "quantize gradients", "op": "quantize", "rows": 8192, "cols": 4096, "in": "bf16",
         "forms": "both", "rounding": "stochastic", "residual": False, "pad": 0},
        # a 4-bit message with error feedback over a bucket of 16M values
        {"name": "quantize message", "op": "quantize", "rows": 4096, "cols": 4096, "in": "f32",
         "forms": "rows", "rounding": "nearest", "residual": True, "pad": 0},
        # activations that are a slice of a wider tensor, ragged both ways, along the tokens
        {"name": "quantize ragged slice", "op": "quantize", "rows": 3001, "cols": 1601,
         "in": "bf16", "forms": "columns", "rounding": "nearest", "residual": False, "pad": 7},
        # one token against the first feed-forward matrix of a GPT-2-XL-shaped block
        {"name": "product one token", "op": "product", "m": 1, "n": 6400, "k": 1600, "out": "bf16",
         "accumulate": False},
        # a handful of sequences against a vocabulary
        {"name": "product vocabulary", "op": "product", "m": 24, "n": 50257, "k": 1600,
         "out": "f32", "accumulate": False},
        # odd in every direction
        {"name": "product ragged", "op": "product", "m": 1000, "n": 777, "k": 1999, "out": "bf16",
         "accumulate": False},
        # weight gradients added up over micro-batches, contraction over 16384 tokens
        {"name": "product accumulate", "op": "product", "m": 4096, "n": 1024, "k": 16384,
         "out": "f32", "accumulate": True},
        # the largest: operations bound it
        {"name": "product large", "op": "product", "m": 8192, "n": 8192, "k": 8192, "out": "bf16",
         "accumulate": False},
        # four tokens through a BERT-Large-shaped feed-forward matrix
        {"name": "linear four tokens", "op": "linear", "tokens": 4, "inner": 1024, "outer": 4096,
         "in": "bf16", "train": False},
        # a training step of the feed-forward matrix of a GPT-2-XL-shaped block, 8192 tokens
        {"name": "linear training", "op": "linear", "tokens": 8192, "inner": 1600, "outer": 6400,
         "in": "bf16", "train": True},
    ]


def _near(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "product", "product", "linear"])
    if op == "quantize":
        residual = rng.random() < 0.25
        rows = _near(rng, 1, 30000)
        return {"op": op, "rows": rows, "cols": _near(rng, 1, min(9000, 33000000 // rows)),
                "in": "f32" if residual else rng.choice(["f32", "bf16"]),
                "forms": "rows" if residual else rng.choice(["rows", "columns", "both"]),
                "rounding": rng.choice(["nearest", "stochastic"]), "residual": residual,
                "pad": rng.choice([0, 0, 0, 1, 8, 13])}
    if op == "product":
        out = rng.choice(["f32", "bf16"])
        return {"op": op, "m": _near(rng, 1, 8192), "n": _near(rng, 1, 8192),
                "k": _near(rng, 1, 8192), "out": out,
                "accumulate": out == "f32" and rng.random() < 0.5}
    return {"op": op, "tokens": _near(rng, 1, 8192), "inner": _near(rng, 16, 1600),
            "outer": _near(rng, 16, 6400), "in": rng.choice(["f32", "bf16"]),
            "train": rng.random() < 0.6}


# ----------------------------------------------------------------------------------------------
# the plain forms

def _power(e):
    """2^e of whole numbers, exactly, in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _mix(x):
    """32 bits mixed into 32 bits; int32 arithmetic that wraps."""
    x = x ^ ((x >> 16) & 0xFFFF)
    x = x * (MIX_A - (1 << 32))
    x = x ^ ((x >> 15) & 0x1FFFF)
    x = x * MIX_B
    return x ^ ((x >> 16) & 0xFFFF)


def _int32(x):
    return ((x + (1 << 31)) & 0xFFFFFFFF) - (1 << 31)


def _random16(total, seed, dev):
    """A 16-bit number for each of total elements (a multiple of 32, below 2^34), from its place
    and the seed."""
    key = torch.full((), _int32(seed + GOLDEN), dtype=torch.int32, device=dev)
    key = _mix(_mix(key) ^ _int32(seed >> 32))
    w = _mix(torch.arange(total // 8, dtype=torch.int32, device=dev) + key)
    weyl = torch.tensor([_int32(j * GOLDEN) for j in range(1, 5)], dtype=torch.int32, device=dev)
    x = w[:, None] + weyl
    x = x ^ ((x >> 15) & 0x1FFFF)
    x = x * _int32(MIX_C)
    x = x ^ ((x >> 16) & 0xFFFF)
    return torch.stack([(x >> 16) & 0xFFFF, x & 0xFFFF], dim=-1).view(-1)


def _quantize(x, rounding, seed):
    """Codes [rows][columns up to a multiple of 32] (uint8, one a byte) and biased exponents
    [rows][blocks] of a matrix in fp32."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    # the smallest exponent with which the largest magnitude does not exceed 6
    e = (x.abs().amax(-1).view(torch.int32) + 0x3FFFFF) >> 23
    e = (e - 2).clamp(min=0)
    z = (x * _power(127 - e)[..., None]).float()
    a = z.abs()
    if rounding == "nearest":              # ties to the even code
        code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
                + (a >= 3.5) + (a > 5))
    else:
        spacing = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        below = torch.floor(a / spacing) * spacing
        chance = torch.floor((a - below) / spacing * 65536).int()
        r = _random16(x.numel(), seed, x.device).view(x.shape)
        below = (below + torch.where(chance + r >= 65536, spacing, 0.0)).clamp(max=6.0)
        code = (below * 2).byte()          # 0 1 2 3 4 6 8 12
        code = torch.where(code < 5, code, 3 + code // 4 + (code > 6).byte())
        code = torch.where(below == 6, 7, torch.where(below == 4, 6, torch.where(
            below == 3, 5, code)))
    code = code | (torch.signbit(z).byte() << 3)
    return code.view(rows, -1), e


def _values(code, e):
    """What codes and biased exponents stand for, in fp32."""
    table = torch.tensor(CODES + tuple(-c for c in CODES), device=code.device)
    v = table[code.int()].view(code.shape[0], -1, BLOCK)
    return (v * _power(e - 127)[..., None]).float().view(code.shape)


def _pack(code, e):
    """Codes two a byte, and the exponents in their tiles."""
    rows, blocks = e.shape
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    rt, bt = -(-rows // 128), -(-blocks // 4)
    t = torch.zeros(rt * 128, bt * 4, dtype=torch.uint8, device=e.device)
    t[:rows, :blocks] = e
    t = t.view(rt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return packed.contiguous(), t


def _unpack(packed, t, rows, cols):
    """What a packed matrix stands for, in fp32."""
    code = torch.stack([packed & 15, packed >> 4], dim=-1).view(rows, -1)
    blocks = code.shape[1] // BLOCK
    rt, bt = -(-rows // 128), -(-blocks // 4)
    e = t.view(rt, bt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, bt * 4)
    return _values(code, e[:rows, :blocks].int())[:, :cols]


def _plain(s):
    case, op = s["case"], s["op"]
    if op == "quantize":
        x, out = s["x"].float(), {}
        if case["residual"]:
            x = x + s["residual"]
        if case["forms"] != "columns":
            v = _values(*_quantize(x, case["rounding"], s["seed"]))[:, :x.shape[1]]
            out["rows"] = v.to(torch.bfloat16)
            if case["residual"]:
                s["residual"].copy_(x - v)
                out["residual"] = s["residual"]
        if case["forms"] != "rows":
            v = _values(*_quantize(x.t().contiguous(), case["rounding"], s["seed"] + 1))
            out["columns"] = v[:, :x.shape[0]].to(torch.bfloat16)
        return out
    if op == "product":
        p = _unpack(*s["a"]) @ _unpack(*s["b"]).t()
        if case["accumulate"]:
            return s["out"].copy_(s["out"] + p)
        return p.to(TYPES[case["out"]])
    x = s["x"].float()

    def rounded(y, rounding="nearest", seed=0):
        return _values(*_quantize(y, rounding, seed))[:, :y.shape[1]]

    out = {"y": (rounded(x) @ _unpack(*s["w"]).t()).to(s["x"].dtype)}
    if case["train"]:
        dy = s["dy"].float()
        out["dx"] = (rounded(dy, "stochastic", s["seed"]) @ _unpack(*s["wt"]).t()).to(s["x"].dtype)
        out["dw"] = rounded(dy.t().contiguous(), "stochastic", s["seed"] + 1) @ rounded(
            x.t().contiguous()).t()
    return out


# ----------------------------------------------------------------------------------------------
# inputs

def _matrix(gen, dev, rows, cols, scale, dtype, pad=0):
    """Normal values; the columns differ in size, a few of them by much, as activations' do. pad:
    a slice of a matrix with that many more columns."""
    size = torch.exp(torch.randn(cols + pad, device=dev, generator=gen) * 0.5)
    size = torch.where(torch.rand(cols + pad, device=dev, generator=gen) < 0.01, 10 * size, size)
    x = torch.randn(rows, cols + pad, device=dev, generator=gen).mul_(size * scale)
    return x.to(dtype)[:, pad // 2:pad // 2 + cols]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op, "seed": 7919 * seed + 1}
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _matrix(gen, dev, rows, cols, 0.02, TYPES[case["in"]], case["pad"])
        if case["residual"]:
            s["residual"] = torch.randn(rows, cols, device=dev, generator=gen) * 0.002
        return s

    def packed(x):                         # a matrix in 4 bits, with its size
        return _pack(*_quantize(x, "nearest", 0)) + tuple(x.shape)

    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = packed(_matrix(gen, dev, m, k, 1.0, torch.float32))
        s["b"] = packed(_matrix(gen, dev, n, k, 0.02, torch.float32))
        if case["accumulate"]:
            s["out"] = torch.randn(m, n, device=dev, generator=gen)
    else:
        t, k, n = case["tokens"], case["inner"], case["outer"]
        w = torch.randn(n, k, device=dev, generator=gen) * 0.02
        s["x"] = _matrix(gen, dev, t, k, 1.0, TYPES[case["in"]])
        s["w"] = packed(w)
        if case["train"]:
            s["wt"] = packed(w.t().contiguous())
            s["dy"] = _matrix(gen, dev, t, n, 1e-3, TYPES[case["in"]])
    if own:                                # the weights as the program holds them
        import communication_compressed_optimizer_momentum_b200 as ob
        if op == "product":
            s["own"] = ob.Mx4(*s["a"]), ob.Mx4(*s["b"])
        else:
            s["own"] = ob.Mx4Linear(w, backward=case["train"])
    return s


# ----------------------------------------------------------------------------------------------
# the library's

def _own(s):
    import communication_compressed_optimizer_momentum_b200 as ob
    case, op = s["case"], s["op"]
    if op == "quantize":
        q = ob.onebit_mx4_quantize(s["x"], forms=case["forms"], rounding=case["rounding"],
                                   seed=s["seed"], residual=s.get("residual"))
        out = {}
        if case["forms"] == "both":
            out["rows"] = ob.onebit_mx4_dequantize(q[0], dtype=torch.bfloat16)
            out["columns"] = ob.onebit_mx4_dequantize(q[1], dtype=torch.bfloat16)
        else:
            out[case["forms"]] = ob.onebit_mx4_dequantize(q, dtype=torch.bfloat16)
        if case["residual"]:
            out["residual"] = s["residual"]
        return out
    if op == "product":
        a, b = s["own"]
        if case["accumulate"]:
            return ob.onebit_mx4_matmul(a, b, out=s["out"], accumulate=True)
        return ob.onebit_mx4_matmul(a, b, dtype=TYPES[case["out"]])
    linear = s["own"]
    if not case["train"]:
        return {"y": linear.forward(s["x"])}
    y, kept = linear.forward(s["x"], keep=True)
    dx, dw = linear.backward(s["dy"], kept, seed=s["seed"])
    return {"y": y, "dx": dx, "dw": dw}


def run(s):
    return _own(s) if own else _plain(s)


def _held(rows, cols):
    """Bytes of a matrix in 4 bits."""
    blocks = -(-cols // BLOCK)
    return rows * blocks * 17


def work(case):
    width, op = {"f32": 4, "bf16": 2}, case["op"]
    if op == "quantize":
        rows, cols, n = case["rows"], case["cols"], case["rows"] * case["cols"]
        b, forms = n * width[case["in"]] + (8 * n if case["residual"] else 0), 0
        # each form is written, and read again for the values that are returned in its place
        for form, held in (("rows", _held(rows, cols)), ("columns", _held(cols, rows))):
            if case["forms"] in (form, "both"):
                b += 2 * held + 2 * n
                forms += 1
        return {"bytes": b, "flops": 6 * n * forms}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        out = m * n * width[case["out"]] * (2 if case["accumulate"] else 1)
        return {"bytes": _held(m, k) + _held(n, k) + out, "flops": 2 * m * n * k}
    t, k, n, w = case["tokens"], case["inner"], case["outer"], width[case["in"]]
    b, f = t * k * w + _held(n, k) + t * n * w, 2 * t * n * k
    if case["train"]:
        b += t * n * w + _held(k, n) + t * k * w + 4 * n * k
        f *= 3
    return {"bytes": b, "flops": f}


# ----------------------------------------------------------------------------------------------
# the definition in 64 bits

def _nearest_or_drawn(x, rounding, seed):
    """A matrix in 64 bits as it is held: the power of two from the largest magnitude's logarithm,
    the grid's spacing from each magnitude's binade; the random numbers in 64-bit integers."""
    rows, cols = x.shape
    low = 0xFFFFFFFF
    x = torch.nn.functional.pad(x, (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    a = x.abs()
    most = a.amax(-1, keepdim=True)
    mantissa, e = torch.frexp(most)        # most = mantissa * 2^e, mantissa in [0.5, 1)
    k = (e - 3 + (mantissa > 0.75)).clamp(min=-127)
    k = torch.where(most > 0, k, -127)
    z = a / _power(k)
    unit = _power((torch.frexp(z).exponent - 1).clamp(min=0) - 1)
    y = z / unit
    if rounding == "nearest":
        y = torch.round(y)
    else:
        def mixed(i):
            i = i ^ (i >> 16)
            i = (i * MIX_A) & low
            i = i ^ (i >> 15)
            i = (i * MIX_B) & low
            return i ^ (i >> 16)

        key = torch.tensor((seed + GOLDEN) & low, device=x.device)
        key = mixed(mixed(key) ^ ((seed >> 32) & low))
        place = torch.arange(x.numel(), device=x.device)
        r = (mixed(((place >> 3) + key) & low) + ((place % 8) // 2 + 1) * GOLDEN) & low
        r = r ^ (r >> 15)
        r = (r * MIX_C) & low
        r = r ^ (r >> 16)
        r = torch.where(place % 2 == 0, r >> 16, r & 0xFFFF)
        y = torch.floor(y + r.view(x.shape).double() / 65536)
    v = y * unit * _power(k)
    return torch.where(x < 0, -v, v).view(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x, out = s["x"].double(), {}
        if case["residual"]:               # the sum is one of fp32 by definition
            x = (x + s["residual"].double()).float().double()
        if case["forms"] != "columns":
            out["rows"] = _nearest_or_drawn(x, case["rounding"], s["seed"])
            if case["residual"]:
                out["residual"] = x - out["rows"]
        if case["forms"] != "rows":
            out["columns"] = _nearest_or_drawn(x.t(), case["rounding"], s["seed"] + 1)
        return out

    def held(packed, tiles, rows, cols):   # place by place
        byte = packed.view(rows, -1).long()
        col = torch.arange(cols, device=byte.device)
        row = torch.arange(rows, device=byte.device)[:, None]
        code = (byte[:, col // 2] >> (4 * (col % 2))) & 15
        field, half = (code % 8) // 2, (code % 2).double()
        v = torch.where(field > 0, (1 + half / 2) * _power(field - 1), half / 2)
        b = col // BLOCK
        tiles_across = -(-(-(-cols // BLOCK)) // 4)
        at = ((row // 128) * tiles_across + b // 4) * 512 + (row % 32) * 16 + (
            row % 128 // 32) * 4 + b % 4
        return torch.where(code > 7, -v, v) * _power(tiles[at].long() - 127)

    if op == "product":
        p = held(*s["a"]) @ held(*s["b"]).t()
        return s["out"].double() + p if case["accumulate"] else p
    x = s["x"].double()
    out = {"y": _nearest_or_drawn(x, "nearest", 0) @ held(*s["w"]).t()}
    if case["train"]:
        dy = s["dy"].double()
        out["dx"] = _nearest_or_drawn(dy, "stochastic", s["seed"]) @ held(*s["wt"]).t()
        out["dw"] = _nearest_or_drawn(dy.t(), "stochastic", s["seed"] + 1) @ _nearest_or_drawn(
            x.t(), "nearest", 0).t()
    return out
