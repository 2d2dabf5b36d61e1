"""Matrices in microscaled 4-bit floating point in plain numpy, 64 bits, from the documented formulas:
place by place where that is quick enough, and written apart from the kernels' way of computing it."""
import numpy as np

BLOCK = 32
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
NAN = 255


def random16(i, seed):
    """The documented 16 random bits of places i."""
    u, M, G = np.uint64, 0xFFFFFFFF, 0x9E3779B9

    def mix(x):
        x = x ^ (x >> u(16))
        x = (x * u(0x9016D2F5)) & u(M)
        x = x ^ (x >> u(15))
        x = (x * u(0x314549A1)) & u(M)
        return x ^ (x >> u(16))
    seed &= (1 << 64) - 1
    key = mix(mix(u((seed + G) & M)) ^ u(seed >> 32))
    i = np.asarray(i, dtype=np.uint64)
    g = i >> u(3)
    w = mix(((g & u(M)) + key + (g >> u(32)) * u(G)) & u(M))
    x = (w + ((i % u(8)) // u(2) + u(1)) * u(G)) & u(M)
    x = x ^ (x >> u(15))
    x = (x * u(0x8A8866C7)) & u(M)
    x = x ^ (x >> u(16))
    return np.where(i % u(2) == 0, x >> u(16), x & u(0xFFFF)).astype(np.int64)


def quantize(x, seed=None, row0=0):
    """(codes, exponents) of a float32 matrix: codes one a byte [rows][32 * blocks], exponents
    [rows][blocks]. seed: None for rounding to nearest. row0: the first row's number."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    full = np.zeros((rows, blocks * BLOCK))
    full[:, :cols] = x
    v = full.reshape(rows, blocks, BLOCK)
    a = np.abs(v)
    most = a.max(axis=2)
    bad = ~(most <= 1.5 * 2.0 ** 127)               # NaN compares false
    with np.errstate(divide="ignore", invalid="ignore"):
        safe = np.where(bad | (most == 0), 1.0, most)
        k = np.ceil(np.log2(safe / 6.0)).astype(np.int64)   # exact enough to be off by one at most
    k = np.where(safe > 6.0 * 2.0 ** k.astype(float), k + 1, k)
    k = np.where(safe <= 6.0 * 2.0 ** (k - 1).astype(float), k - 1, k)
    k = np.where(most == 0, -127, np.maximum(k, -127))
    z = np.where(bad[..., None], 0.0, a / 2.0 ** np.where(bad, 0, k)[..., None].astype(float))
    z = np.where(bad[..., None], 0.0, z)
    low = np.searchsorted(VALUES, z, side="right") - 1
    low = np.minimum(low, 7)
    high = np.minimum(low + 1, 7)
    gap = np.where(high > low, VALUES[high] - VALUES[low], 1.0)
    r = (z - VALUES[low]) / gap
    if seed is None:
        up = (r > 0.5) | ((r == 0.5) & (low % 2 == 1))
    else:
        place = np.arange(rows * blocks * BLOCK, dtype=np.int64).reshape(z.shape)
        place = place + row0 * blocks * BLOCK
        up = np.floor(65536 * r) + random16(place, seed) >= 65536
    code = np.where(up, high, low)
    # the sign of what is rounded to zero stays
    code = code + 8 * (np.signbit(v) & ~bad[..., None])
    e = np.where(bad, NAN, k + 127)
    return code.reshape(rows, -1).astype(np.uint8), e.astype(np.uint8)


def values(code, e, cols):
    """What codes and exponents stand for."""
    rows, blocks = e.shape
    v = np.where(code > 7, -1.0, 1.0) * VALUES[code & 7]
    v = v.reshape(rows, blocks, BLOCK) * 2.0 ** (e.astype(np.int64) - 127)[..., None].astype(float)
    v = np.where((e == NAN)[..., None], np.nan, v)
    return v.reshape(rows, -1)[:, :cols]


def pack(code, e):
    """The documented bytes: (codes [rows][16 * blocks], scales flat)."""
    rows, blocks = e.shape
    packed = (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    across = -(-blocks // 4)
    scales = np.zeros(-(-rows // 128) * across * 512, dtype=np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    at = ((r // 128) * across + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
    scales[at] = e
    return packed, scales
