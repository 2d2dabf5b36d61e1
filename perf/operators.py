"""The optimizer operators over many tensors, as they are measured: an AdamW step with 32-bit
states, the same step with 8-bit states, the global gradient norm with its clip factor, and the
way in and out of the 8-bit states.

``run`` computes them in elementary torch operations, or, where ``own`` is true, makes the calls
a user makes of the library. Parameters, gradients and copies are lists of tensors; the states
of all tensors lie in one flat vector, each tensor's part padded to whole blocks of 256 elements.
"""
import math
import random

import torch

own = False

LR, BETA1, BETA2, EPS, DECAY = 1e-4, 0.9, 0.999, 1e-8, 0.01
BLOCK = 256                       # elements of a tensor that share one exponent in the 8-bit states
GOLDEN, MIX_A, MIX_B, MIX_C = 0x9E3779B9, 0x9016D2F5, 0x314549A1, 0x8A8866C7
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------------------------
# the cases

def _sizes(case):
    """The tensors' lengths. "blocks": transformer blocks and an embedding; "vectors": only the
    biases and norms of the blocks (the group without weight decay); "flat": one tensor;
    "ragged": lengths of every kind between lo and hi, one of them empty."""
    kind = case["tensors"]
    if kind == "flat":
        return [case["numel"]]
    if kind == "ragged":
        r = random.Random(case["pick"])
        lo, hi = math.log(case["lo"]), math.log(case["hi"])
        return [0] + [int(math.exp(r.uniform(lo, hi))) for _ in range(case["count"])]
    h, f = case["hidden"], case["ffn"]
    vectors = [h, h, h, h, f, h, h, h, h, h]
    matrices = [h * h, h * h, h * h, h * h, h * f, h * f]
    if kind == "vectors":
        return vectors * case["layers"]
    return (matrices + vectors) * case["layers"] + [case["vocab"] * h]


def listed():
    large = {"tensors": "blocks", "layers": 24, "hidden": 1024, "ffn": 4096, "vocab": 30522}
    xl = {"tensors": "blocks", "layers": 48, "hidden": 1600, "ffn": 6400, "vocab": 50257}
    return [
        # biases and norms of a BERT-Large-shaped model, their own group: latency of one small call
        {"name": "adamw vectors", "op": "adamw", "param": "f32", "grad": "f32", "copy": False,
         "align": 64, "tensors": "vectors", "layers": 24, "hidden": 1024, "ffn": 4096},
        # one bucket of a million parameters
        {"name": "adamw bucket 1M", "op": "adamw", "param": "f32", "grad": "f32", "copy": False,
         "align": 64, "tensors": "flat", "numel": 1048576},
        # mixed-precision training: fp32 master weights, bf16 gradients, bf16 copy for the forward
        {"name": "adamw bert-large", "op": "adamw", "param": "f32", "grad": "bf16", "copy": True,
         "align": 64, **large},
        # views of a flat buffer, back to back at odd offsets, pure bf16
        {"name": "adamw ragged views", "op": "adamw", "param": "bf16", "grad": "bf16",
         "copy": False, "align": 1, "tensors": "ragged", "count": 500, "lo": 1, "hi": 500000,
         "pick": 11},
        {"name": "adamw8 bucket 1M", "op": "adamw8", "param": "f32", "grad": "f32", "copy": False,
         "align": 64, "tensors": "flat", "numel": 1048576},
        {"name": "adamw8 bert-large", "op": "adamw8", "param": "f32", "grad": "bf16",
         "copy": True, "align": 64, **large},
        # the largest model whose whole training state is meant to fit: pure bf16, 8-bit states
        {"name": "adamw8 gpt2-xl", "op": "adamw8", "param": "bf16", "grad": "bf16",
         "copy": False, "align": 64, **xl},
        {"name": "adamw8 ragged views", "op": "adamw8", "param": "f32", "grad": "f32",
         "copy": False, "align": 1, "tensors": "ragged", "count": 300, "lo": 1, "hi": 300000,
         "pick": 12},
        {"name": "norm vectors", "op": "norm", "grad": "f32", "align": 64, "tensors": "vectors",
         "layers": 24, "hidden": 1024, "ffn": 4096},
        {"name": "norm gpt2-xl", "op": "norm", "grad": "bf16", "align": 64, **xl},
        # a checkpoint written from, and read into, the 8-bit states
        {"name": "get state bert-large", "op": "get", "out": "f32", **large},
        {"name": "set state ragged", "op": "set", "tensors": "ragged", "count": 300, "lo": 1,
         "hi": 300000, "pick": 13},
    ]


def _near(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "adamw8", "adamw8", "norm", "get", "set"])
    case = {"op": op}
    if op in ("adamw", "adamw8"):
        case["param"] = rng.choice(["f32", "bf16"])
        case["copy"] = case["param"] == "f32" and rng.random() < 0.4
    if op in ("adamw", "adamw8", "norm"):
        case["grad"] = rng.choice(["f32", "bf16"])
        case["align"] = rng.choice([1, 2, 8, 64, 64])
    if op == "get":
        case["out"] = rng.choice(["f32", "bf16"])
    kind = rng.choice(["flat", "blocks", "vectors", "ragged"])
    case["tensors"] = kind
    if kind == "flat":
        case["numel"] = _near(rng, 1, 200000000)
    elif kind == "ragged":
        case.update(count=_near(rng, 1, 1500), lo=1, hi=_near(rng, 50, 400000),
                    pick=rng.randrange(1 << 30))
    else:
        h = _near(rng, 60, 1100)
        case.update(layers=_near(rng, 1, 24), hidden=h, ffn=4 * h)
        if kind == "blocks":
            case["vocab"] = _near(rng, 100, 30000)
    return case


def _padded(sizes):
    return [-(-n // BLOCK) * BLOCK for n in sizes]


# ----------------------------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    sizes = _sizes(case)
    padded = _padded(sizes)
    total = sum(padded)
    lengths = torch.tensor(padded, device=dev)
    s = {"case": case, "sizes": sizes, "padded": padded, "op": case["op"]}

    def normal(n, scale, dtype=torch.float32):
        x = torch.randn(n, device=dev, generator=gen)
        return (x.mul_(scale) if scale is not None else x).to(dtype)

    # gradients of one tensor are of one size; the tensors' sizes go over two decades
    sigma = 10.0 ** (torch.rand(len(sizes), device=dev, generator=gen) * 2 - 4)
    if case["op"] in ("adamw", "adamw8", "norm"):
        align = case["align"]
        room = [-(-n // align) * align for n in sizes]
        at = [0]
        for n in room:
            at.append(at[-1] + n)
        spread = torch.repeat_interleave(sigma, torch.tensor(room, device=dev),
                                         output_size=at[-1])
        g = normal(at[-1], spread, TYPES[case["grad"]])
        del spread
        s["grads"] = [g[a:a + n] for a, n in zip(at, sizes)]
        if case["op"] == "norm":
            s["max_norm"] = 1.0
            s["work"] = torch.zeros(16384, dtype=torch.uint8, device=dev)
            return s
        p = normal(at[-1], 0.02, TYPES[case["param"]])
        s["params"], s["param_arena"] = [p[a:a + n] for a, n in zip(at, sizes)], p
        s["copies"] = None
        if case["copy"]:
            c = p.to(torch.bfloat16)
            s["copies"], s["copy_arena"] = [c[a:a + n] for a, n in zip(at, sizes)], c
        # matrices decay, vectors do not; the scale is what a clipped step brings along
        s["decay"] = [DECAY if n > 65536 else 0.0 for n in sizes]
        s["scale"] = torch.rand(1, device=dev, generator=gen) * 0.5 + 0.5
        t = 40 + seed % 20
        ctl = torch.zeros(8, dtype=torch.int64)
        ctl[0] = t
        ctl[2:4] = torch.tensor([1 - BETA1 ** t, 1 - BETA2 ** t], dtype=torch.float64).view(
            torch.int64)
        s["ctl"] = ctl.to(dev)
        s["seed"] = 7919 * seed + 1

    spread = torch.repeat_interleave(sigma, lengths, output_size=total)
    m = normal(total, 0.3).mul_(spread)
    v = torch.rand(total, device=dev, generator=gen).add_(0.02).mul_(spread).mul_(spread)
    # the places behind a tensor are zero, and stay so
    start = torch.tensor([0] + padded[:-1], device=dev).cumsum(0)
    place = torch.arange(total, device=dev) - torch.repeat_interleave(start, lengths,
                                                                      output_size=total)
    inside = place < torch.repeat_interleave(torch.tensor(sizes, device=dev), lengths,
                                             output_size=total)
    m.mul_(inside)
    v.mul_(inside)
    del spread, place, inside
    if case["op"] in ("adamw", "set"):
        s["m"], s["v"] = m, v
        if case["op"] == "adamw":
            return s
    if case["op"] == "set":
        s["m_codes"], s["v_codes"] = (torch.zeros(total, dtype=torch.uint8, device=dev)
                                      for _ in range(2))
        s["m_exp"], s["v_exp"] = (torch.zeros(total // BLOCK, dtype=torch.uint8, device=dev)
                                  for _ in range(2))
        return s
    s["m_codes"], s["m_exp"] = _encode(m, None, True)
    del m
    s["v_codes"], s["v_exp"] = _encode(v, None, False)
    return s


# ----------------------------------------------------------------------------------------------
# the plain forms

def _power(e):
    """2^e of whole numbers, exactly, in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _encode(x, random_bits, signed):
    """Codes and exponents of a vector of whole blocks. The block's exponent is the smallest
    whose largest code holds every value; each value is scaled by a power of two, so that its
    code is the upper bits of its fp32 pattern, and rounded there: to the nearest, ties to even,
    or up with the probability that 20 random bits give."""
    top = 15 if signed else 31
    a = (x.abs() if signed else x.clamp(min=0)).view(-1, BLOCK)
    k = (a.amax(1).view(torch.int32) + 0xFFFFF) >> 23
    z = (a * _power(top - k)[:, None]).float().view(-1).view(torch.int32)
    add = random_bits if random_bits is not None else 0x7FFFF + ((z >> 20) & 1)
    code = (z + add) >> 20
    if signed:
        code = code | ((x < 0).int() << 7)
    else:
        code = torch.maximum(code, (x > 0).int())
    return code.to(torch.uint8), k.to(torch.uint8)


def _decode(codes, exps, signed):
    top = 15 if signed else 31
    c = codes.view(-1, BLOCK).int()
    a = ((c & 127 if signed else c) << 20).view(torch.float32)
    x = (a * _power(exps.int() - top)[:, None]).float()
    if signed:
        x = torch.where(c > 127, -x, x)
    return x.view(-1)


def _mix(x):
    """32 bits mixed into 32 bits; int32 arithmetic that wraps."""
    x = x ^ ((x >> 16) & 0xFFFF)
    x = x * (MIX_A - (1 << 32))
    x = x ^ ((x >> 15) & 0x1FFFF)
    x = x * MIX_B
    return x ^ ((x >> 16) & 0xFFFF)


def _int32(x):
    return ((x + (1 << 31)) & 0xFFFFFFFF) - (1 << 31)


def _random_bits(total, seed, t):
    """Two 20-bit numbers for each element, from its place, the seed and the step's number."""
    key = torch.full((), _int32(seed + GOLDEN), dtype=torch.int32, device=t.device)
    key = _mix(_mix(key) ^ _int32(seed >> 32))
    key = _mix(key + t.int())
    w = _mix(torch.arange(total // 8, dtype=torch.int32, device=t.device) + key)
    weyl = torch.arange(1, 9, dtype=torch.int32, device=t.device) * _int32(GOLDEN)
    x = (w[:, None] + weyl).view(-1)
    x = x ^ ((x >> 15) & 0x1FFFF)
    x = x * _int32(MIX_C)
    x = x ^ ((x >> 16) & 0xFFFF)
    return (x >> 12) & 0xFFFF0, (x & 0xFFFF) << 4


def _flat(tensors, padded, zeros):
    """The tensors one after another in fp32, each padded with zeros to whole blocks."""
    return torch.cat([y for x, n in zip(tensors, padded) for y in (x, zeros[:n - x.numel()])]
                     ).float()


def _plain_step(s):
    dev = s["ctl"].device
    padded = s["padded"]
    eight = s["op"] == "adamw8"
    s["ctl"][0].add_(1)
    c = s["ctl"].view(torch.float64)[2:4]
    c.mul_(torch.tensor([BETA1, BETA2], dtype=torch.float64, device=dev)).add_(
        torch.tensor([1 - BETA1, 1 - BETA2], dtype=torch.float64, device=dev))
    step = (LR / c[0]).float()
    r2 = (1 / c[1].sqrt()).float()
    grad_type = s["grads"][0].dtype
    g = _flat(s["grads"], padded, torch.zeros(BLOCK, dtype=grad_type, device=dev)) * s["scale"]
    m = _decode(s["m_codes"], s["m_exp"], True) if eight else s["m"]
    v = _decode(s["v_codes"], s["v_exp"], False) if eight else s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    del g
    if eight:
        rm, rv = _random_bits(m.numel(), s["seed"], s["ctl"][0])
        codes, exps = _encode(m, rm, True)
        s["m_codes"].copy_(codes)
        s["m_exp"].copy_(exps)
        codes, exps = _encode(v, rv, False)
        s["v_codes"].copy_(codes)
        s["v_exp"].copy_(exps)
        del rm, rv, codes
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    update = step * (m / (v.sqrt() * r2 + EPS))
    del m, v
    keep = torch.repeat_interleave(
        1 - LR * torch.tensor(s["decay"], dtype=torch.float64, device=dev),
        torch.tensor(padded, device=dev), output_size=update.numel()).float()
    param_type = s["params"][0].dtype
    p = _flat(s["params"], padded, torch.zeros(BLOCK, dtype=param_type, device=dev))
    p = p * keep - update
    del keep, update
    new = [x[:n] for x, n in zip(p.split(padded), s["sizes"])]
    torch._foreach_copy_(s["params"], new)
    if s["copies"] is not None:
        torch._foreach_copy_(s["copies"], new)
    out = {"params": s["param_arena"], "count": s["ctl"][0]}
    if s["copies"] is not None:
        out["copies"] = s["copy_arena"]
    if eight:
        out["m"] = _decode(s["m_codes"], s["m_exp"], True).to(torch.bfloat16)
        out["v"] = _decode(s["v_codes"], s["v_exp"], False).to(torch.bfloat16)
    else:
        out["m"], out["v"] = s["m"], s["v"]
    return out


def _plain(s):
    op = s["op"]
    if op in ("adamw", "adamw8"):
        return _plain_step(s)
    if op == "norm":
        norm = torch.cat(s["grads"]).double().square().sum().sqrt()
        scale = torch.clamp(s["max_norm"] / norm, max=1.0)
        return {"norm": norm.float(), "scale": scale.float()}
    if op == "get":
        dtype = TYPES[s["case"]["out"]]
        return {"m": _decode(s["m_codes"], s["m_exp"], True).to(dtype),
                "v": _decode(s["v_codes"], s["v_exp"], False).to(dtype)}
    codes, exps = _encode(s["m"], None, True)
    s["m_codes"].copy_(codes)
    s["m_exp"].copy_(exps)
    codes, exps = _encode(s["v"], None, False)
    s["v_codes"].copy_(codes)
    s["v_exp"].copy_(exps)
    return {"m": _decode(s["m_codes"], s["m_exp"], True).to(torch.bfloat16),
            "v": _decode(s["v_codes"], s["v_exp"], False).to(torch.bfloat16)}


# ----------------------------------------------------------------------------------------------
# the library's

def _own(s):
    import communication_compressed_optimizer_momentum_b200 as ob
    op = s["op"]
    if op == "norm":
        norm, scale = ob.onebit_grad_norm(s["grads"], s["max_norm"], work=s["work"])
        return {"norm": norm, "scale": scale}
    if op == "adamw":
        ob.onebit_adamw_step(s["params"], s["grads"], s["m"], s["v"], s["ctl"], LR, BETA1, BETA2,
                             EPS, s["decay"], copies=s["copies"], grad_scale=s["scale"])
        out = {"params": s["param_arena"], "count": s["ctl"][0], "m": s["m"], "v": s["v"]}
    else:
        state = (s["m_codes"], s["v_codes"], s["m_exp"], s["v_exp"])
        if op == "get":
            m, v = ob.onebit_adamw8_get_state(*state, dtype=TYPES[s["case"]["out"]])
            return {"m": m, "v": v}
        if op == "set":
            ob.onebit_adamw8_set_state(*state, s["m"], s["v"])
            m, v = ob.onebit_adamw8_get_state(*state, dtype=torch.bfloat16)
            return {"m": m, "v": v}
        ob.onebit_adamw8_step(s["params"], s["grads"], *state, s["ctl"], LR, BETA1, BETA2, EPS,
                              s["decay"], copies=s["copies"], grad_scale=s["scale"],
                              seed=s["seed"])
        m, v = ob.onebit_adamw8_get_state(*state, dtype=torch.bfloat16)
        out = {"params": s["param_arena"], "count": s["ctl"][0], "m": m, "v": v}
    if s["copies"] is not None:
        out["copies"] = s["copy_arena"]
    return out


def run(s):
    return _own(s) if own else _plain(s)


def work(case):
    sizes = _sizes(case)
    n, total, op = sum(sizes), sum(_padded(sizes)), case["op"]
    width = {"f32": 4, "bf16": 2}
    if op == "norm":
        return {"bytes": n * width[case["grad"]] + 8, "flops": 2 * n}
    # 8-bit states are returned as the values they stand for: read once more, written out
    values = total * (2 + 2 * width[case.get("out", "bf16")]) + total // BLOCK * 2
    if op == "get":
        return {"bytes": values, "flops": 2 * total}
    if op == "set":
        return {"bytes": total * 10 + total // BLOCK * 2 + values, "flops": 8 * total}
    each = 2 * width[case["param"]] + width[case["grad"]] + (2 if case["copy"] else 0)
    if op == "adamw":
        return {"bytes": n * (each + 16), "flops": 15 * n}
    return {"bytes": n * (each + 4) + total // BLOCK * 4 + values, "flops": 30 * n}


# ----------------------------------------------------------------------------------------------
# the definition in 64 bits

def exact(case, seed):
    """Tensor by tensor in 64 bits. A code's value is found by its binade and the rounding within
    it; the random numbers are whole numbers, worked out in 64-bit integers."""
    sizes = _sizes(case)
    if sum(sizes) > 700_000_000 and case["op"] != "norm":
        return None
    s = prepare(case, seed)
    dev = torch.device("cuda", torch.cuda.current_device())
    low = 0xFFFFFFFF
    if case["op"] == "norm":
        total = 0.0
        for g in s["grads"]:
            total += float(g.double().pow(2).sum()) if g.numel() else 0.0
        norm = math.sqrt(total)
        return {"norm": torch.tensor(norm, dtype=torch.float64),
                "scale": torch.tensor(min(1.0, s["max_norm"] / norm) if norm else 1.0,
                                      dtype=torch.float64)}

    def value(codes, exps, bits):          # of a code with `bits` exponent bits and 3 others
        c = codes.view(-1, BLOCK).long()
        sign = torch.where(c >= 128, -1.0, 1.0).double() if bits == 4 else 1.0
        c = c % 128 if bits == 4 else c
        field, rest = c // 8, (c % 8).double() / 8
        top = 2 ** bits - 1
        size = torch.where(field > 0, (1 + rest) * _power(field - top), rest * 2.0 ** (1 - top))
        return (sign * size * _power(exps.long() - 127)[:, None]).view(-1)

    def rounded(x, chance, bits):          # the value that x is held as; chance: None, or in [0, 1)
        a = x.abs().view(-1, BLOCK)
        most = a.amax(1)
        e = torch.frexp(most).exponent - 1
        e = (e + (most > 1.875 * _power(e)).int()).clamp(min=-127)[:, None]
        least = (e - 2 ** bits + 2)        # the binade below which the steps stay the same
        unit = _power(torch.maximum(torch.frexp(a).exponent - 1, least) - 3)
        y = a / unit
        y = torch.round(y) if chance is None else torch.floor(y + chance.view(-1, BLOCK))
        if bits == 5:
            y = torch.where((y == 0) & (a > 0), 1.0, y)
        return torch.where(x.view(-1, BLOCK) < 0, -(y * unit), y * unit).view(-1)

    if case["op"] == "get":
        return {"m": value(s["m_codes"], s["m_exp"], 4), "v": value(s["v_codes"], s["v_exp"], 5)}
    if case["op"] == "set":
        return {"m": rounded(s["m"].double(), None, 4), "v": rounded(s["v"].double(), None, 5)}

    def mixed(x):
        x = x ^ (x >> 16)
        x = (x * MIX_A) & low
        x = x ^ (x >> 15)
        x = (x * MIX_B) & low
        return x ^ (x >> 16)

    t = int(s["ctl"][0]) + 1
    key = mixed(mixed((s["seed"] + GOLDEN) & low) ^ ((s["seed"] >> 32) & low))
    key = mixed((key + t) & low)
    c1, c2 = 1 - BETA1 ** t, 1 - BETA2 ** t
    out = {"params": s["param_arena"].double(), "count": None}
    if s["copies"] is not None:
        out["copies"] = s["copy_arena"].double()
    eight = case["op"] == "adamw8"
    if not eight:
        out["m"], out["v"] = s["m"].double(), s["v"].double()
    else:
        out["m"], out["v"] = (torch.empty(s["m_codes"].numel(), dtype=torch.float64, device=dev)
                              for _ in range(2))
    scale = s["scale"].double()
    at = 0
    for i, (n, whole) in enumerate(zip(s["sizes"], s["padded"])):
        if n == 0:
            continue
        b = slice(at // BLOCK, (at + whole) // BLOCK)
        if eight:
            held = [value(s[c][at:at + whole], s[k][b], bits)
                    for c, k, bits in (("m_codes", "m_exp", 4), ("v_codes", "v_exp", 5))]
        else:
            held = [out["m"][at:at + whole], out["v"][at:at + whole]]
        g = s["grads"][i].double() * scale
        m = BETA1 * held[0][:n] + (1 - BETA1) * g
        v = BETA2 * held[1][:n] + (1 - BETA2) * g * g
        p = s["params"][i].double() * (1 - LR * s["decay"][i])
        p = p - LR * (m / c1) / (torch.sqrt(v / c2) + EPS)
        first = s["params"][i].storage_offset()
        out["params"][first:first + n] = p
        if s["copies"] is not None:
            out["copies"][first:first + n] = p
        if eight:
            place = torch.arange(at, at + whole, device=dev)
            x = (mixed(((place >> 3) + key) & low) + (place % 8 + 1) * GOLDEN) & low
            x = x ^ (x >> 15)
            x = (x * MIX_C) & low
            x = x ^ (x >> 16)
            for name, y, r, bits in (("m", m, x >> 16, 4), ("v", v, x & 0xFFFF, 5)):
                y = torch.nn.functional.pad(y, (0, whole - n))
                y = rounded(y, r.double() / 65536, bits)
                out[name][at:at + whole] = y
        else:
            out["m"][at:at + n], out["v"][at:at + n] = m, v
        at += whole
    return out
