"""AdamW over a list of tensors in 64 bits, and how far an fp32 evaluation of it may be off: the
plain implementation that the GPU tests compare with. numpy only.

Error bounds: u = 2^-24 is the largest relative error of one fp32 rounding; every bound is the sum
over the operations of the step in the order they are done, to first order, times 1.01 for the
higher ones, plus a few of fp32's smallest subnormals for results below the normal range."""
import numpy as np

BLOCK = 256
U = 2.0 ** -24
TINY = 2.0 ** -149
TOP_M, TOP_V = 15, 31


def fp32(x):
    return np.asarray(x, dtype=np.float32)


def corrections(t, beta1, beta2, on=True):
    return (1 - beta1 ** t, 1 - beta2 ** t) if on else (1.0, 1.0)


def step64(p, g, m, v, t, lr, beta1, beta2, eps, wd, scale=1.0, bias=True):
    """One step on float64 arrays: (p, m, v) after it, and a bound for each on an fp32 evaluation's
    error."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    with np.errstate(all="ignore"):
        gs = g * scale                                  # fp32: 1 rounding
        parts_m = np.abs(beta1 * m) + np.abs((1 - beta1) * gs)
        m1 = beta1 * m + (1 - beta1) * gs
        # coefficient, product, sum, and the gradient's own rounding
        em = 4 * U * parts_m * 1.01 + 4 * TINY
        v1 = beta2 * v + (1 - beta2) * gs * gs
        # coefficient, square, product, sum, and twice the gradient's own
        ev = 6 * U * v1 * 1.01 + 4 * TINY
        c1, c2 = corrections(t, beta1, beta2, bias)
        root = np.sqrt(v1 / c2)
        den = root + eps
        # v's error halves under the root (or is all of it near 0), then root, 1/sqrt(c2), product
        er = np.minimum(ev / 2 / np.maximum(np.sqrt(v1), 1e-300), np.sqrt(ev)) / np.sqrt(c2) \
            + 3 * U * root
        ed = er + 2 * U * den                           # eps' rounding and the sum's
        q = m1 / den
        # m's error, the denominator's, the division
        eq = em / den + np.abs(q) * ed / np.maximum(den - ed, 1e-300) + U * np.abs(q) + TINY
        upd = lr / c1 * q
        eu = lr / c1 * eq + 2 * U * np.abs(upd)         # lr / c1, product
        p1 = p * (1 - lr * wd) - upd
        ep = 1.01 * (eu + 2 * U * np.abs(p) + U * np.abs(p1)) + 4 * TINY
    return (p1, m1, v1), (ep, em, ev)


def bf16_bound(x, err):
    """The same after one rounding to bf16: half a step is at most 2^-8 of the value."""
    return err + 2.0 ** -8 * (np.abs(x) + err) + 2.0 ** -134


def random_words(i, seed, t):
    """The documented 32 random bits of state elements i at step t (uint32)."""
    u, M = np.uint64, 0xFFFFFFFF
    G = 0x9E3779B9

    def mix(x):
        x = x ^ (x >> u(16))
        x = (x * u(0x9016D2F5)) & u(M)
        x = x ^ (x >> u(15))
        x = (x * u(0x314549A1)) & u(M)
        return x ^ (x >> u(16))
    key = mix(u((seed + G) & M))
    key = mix(key ^ u((seed >> 32) & M))
    key = mix((key + u(t & M)) & u(M))
    i = np.asarray(i, dtype=np.uint64)
    g = i >> u(3)
    w = mix(((g & u(M)) + key + (g >> u(32)) * u(G)) & u(M))
    x = (w + (i % u(8) + u(1)) * u(G)) & u(M)
    x = x ^ (x >> u(15))
    x = (x * u(0x8A8866C7)) & u(M)
    return (x ^ (x >> u(16))).astype(np.uint32)


def decode64(codes, exps, signed):
    """The values of codes [blocks * 256] with exponents [blocks], from the documented formula."""
    c = np.asarray(codes).reshape(-1, BLOCK).astype(np.int64)
    top = TOP_M if signed else TOP_V
    a = c & 127 if signed else c
    f = np.where(a < 8, np.ldexp(a / 8.0, 1 - top), np.ldexp(1 + (a % 8) / 8.0, a // 8 - top))
    k = np.asarray(exps).astype(np.int64)[:, None]
    x = np.where(k == 255, np.nan, np.ldexp(f, k - 127))
    return np.where(signed & (c > 127), -x, x).reshape(-1)


def exponents64(x):
    """The exponent of each block of 256 fp32 values (float64 arrays that hold them)."""
    a = np.abs(np.asarray(x, np.float64)).reshape(-1, BLOCK)
    most = a.max(1)
    finite = np.isfinite(most)
    with np.errstate(all="ignore"):
        e = np.frexp(np.where(finite, most, 1.0))[1] - 1
        e = np.where(most > 1.875 * np.ldexp(1.0, e), e + 1, e)
        # below the normal range every window has the steps of fp32's subnormals
        e = np.maximum(e, -127)
        sub = most < 2.0 ** -126
        e = np.where(sub, np.where(most > 1.75 * 2.0 ** -127, -126, -127), e)
    return np.where(finite & (e < 128), e + 127, 255).astype(np.int64)


def encode64(x, signed, chance=None):
    """Codes and exponents of fp32 values x (whole blocks): rounded to nearest even, or up with the
    probabilities that chance in [0, 1) decides."""
    x = np.asarray(x, np.float64)
    top = TOP_M if signed else TOP_V
    k = exponents64(x)
    a = np.abs(x).reshape(-1, BLOCK)
    a = np.where((k == 255)[:, None], 0.0, a)
    # z is the value below a common power of two; where it is below fp32's normal range it is
    # itself rounded to a multiple of 2^-149, 2^20 times finer than a code
    z = np.ldexp(a, (top - k)[:, None]).astype(np.float32).view(np.uint32).astype(np.int64)
    if chance is None:
        c = (z + 0x7FFFF + ((z >> 20) & 1)) >> 20
    else:
        r = np.round(np.asarray(chance) * 65536).astype(np.int64).reshape(-1, BLOCK) << 4
        c = (z + r) >> 20
    if signed:
        c = c | np.where(np.signbit(x).reshape(-1, BLOCK), 128, 0)
    else:
        c = np.maximum(c, (a > 0).astype(np.int64))
    c = np.where((k == 255)[:, None], 0, c)
    return c.reshape(-1).astype(np.uint8), k.astype(np.uint8)


def moments32(g, m, v, beta1, beta2, scale=1.0):
    """m and v after the step, each fp32 operation rounded as documented (numpy's fp32 is IEEE)."""
    f = np.float32
    with np.errstate(all="ignore"):
        gs = fp32(g) * f(scale)
        m1 = f(beta1) * fp32(m) + f(1 - beta1) * gs
        v1 = f(beta2) * fp32(v) + f(1 - beta2) * (gs * gs)
    return m1, v1
