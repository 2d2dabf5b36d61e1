"""Products of matrices in microscaled 4-bit floating point at every width of the kernel's tiles, for
results that leave by TMA and for others, with values whose sums nothing rounds."""
import ctypes

import pytest
import torch

import communication_compressed_optimizer_momentum_b200 as ob
from communication_compressed_optimizer_momentum_b200 import _abi

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def tiles(m, n, k, dtype):
    """(rows of a tile of out, blocks that share its common axis) of a product; 0 rows: no tensor
    cores."""
    rows, split = ctypes.c_int32(), ctypes.c_int32()
    f = _abi.lib().onebit_internal_mx4_tiles
    f.restype = None
    f(*(ctypes.c_int64(x) for x in (m, n, k)), ctypes.c_int32(0 if dtype == F32 else 1),
      ctypes.byref(rows), ctypes.byref(split))
    return rows.value, split.value


def held(rows, cols, seed):
    """Values that 4 bits hold, in 4 bits and in 64 bits: multiples of 1/2 up to 6."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    v = table[torch.randint(0, 8, (rows, cols), device=DEV, generator=gen)]
    v = v * (torch.randint(0, 2, (rows, cols), device=DEV, generator=gen) * 2 - 1)
    q = ob.onebit_mx4_quantize(v)
    assert torch.equal(ob.onebit_mx4_dequantize(q), v)
    return q, v.double()


# m, n, k, and the tiles of fp32 and of bf16 results. Up to 11 tiles a thread block, so that both
# accumulators are used again; up to 16 stages of the common axis; last tiles of part of the rows and of
# the columns. bf16 rows leave by TMA where n is a multiple of 8, fp32 ones where it is one of 4.
EXACT = [(1, 4096, 1024, (0, 1), (0, 1)), (4, 3001, 1000, (0, 1), (0, 1)), (3, 1000, 99, (0, 1), (0, 1)),
         (13, 2000, 5000, (16, 5), (16, 5)), (16, 40000, 300, (16, 1), (16, 1)),
         (30, 3000, 4000, (32, 4), (32, 4)), (31, 3001, 4000, (32, 4), (32, 4)),
         (32, 30000, 600, (32, 1), (32, 1)), (200, 3000, 1000, (64, 1), (64, 1)),
         (201, 3003, 1000, (64, 1), (64, 1)), (1030, 1104, 3000, (128, 1), (128, 1)),
         (5000, 5008, 1000, (128, 1), (256, 1)), (4100, 4000, 4000, (256, 1), (256, 1)),
         (4100, 4004, 2000, (256, 1), (256, 1)), (4001, 3999, 2000, (256, 1), (256, 1)),
         (2800, 2616, 700, (128, 1), (128, 1)), (2800, 2617, 700, (128, 1), (128, 1))]


@pytest.mark.parametrize("m,n,k,wide,narrow", EXACT)
def test_exact_products_of_every_tile(m, n, k, wide, narrow):
    """All products are multiples of 1/4 and no sum of magnitudes exceeds 36 * 5000: every fp32 sum is
    exact, and bf16 rounds it once. All of out is compared, and what lies beside it stays."""
    assert (tiles(m, n, k, F32), tiles(m, n, k, BF16)) == (wide, narrow)
    (qa, a), (qb, b) = held(m, k, 1), held(n, k, 2)
    want = a @ b.t()
    for dtype in (F32, BF16):
        room = torch.full((m + 2, n + 16), 3.0, device=DEV, dtype=dtype)
        for start in (8, 3):               # rows of the slice begin at 16 bytes (where n + 16 allows), or not
            out = room[1:-1, start:start + n]
            ob.onebit_mx4_matmul(qa, qb, out=out)
            assert torch.equal(out, want.to(dtype))
            out.fill_(3.0)
            assert (room == 3.0).all()
        assert torch.equal(ob.onebit_mx4_matmul(qa, qb, dtype=dtype), want.to(dtype))
    base = torch.randint(-99, 99, (m, n), device=DEV).float()
    assert torch.equal(ob.onebit_mx4_matmul(qa, qb, out=base.clone(), accumulate=True),
                       (base + want).float())
    assert ob.onebit_mx4_status() == 0


@pytest.mark.parametrize("m", [1, 2, 4, 5, 40])
def test_sums_beyond_the_range_of_fp32(m):
    """Blocks whose products cancel but for one, +-1/4 times a power of two: the result is that value as
    fp32 holds it, infinity from 2^128 on, and 0 where all of them cancel, with and without tensor cores
    and for plain values."""
    x = torch.zeros(m, 70, device=DEV)
    w = torch.zeros(40, 70, device=DEV)
    for i, at in enumerate((0, 32)):
        x[:, at:at + 3] = torch.tensor([6, 6, 0.5], device=DEV)
        for r, last in enumerate((0.5, -0.5, 0.0)):
            w[r, at:at + 3] = torch.tensor([6, -6, last if i == 0 else 0], device=DEV)
    for ex, ew in ((120, 12), (120, 10), (120, 9), (10, 119), (124, 124), (-126, 124), (60, 70), (0, 0)):
        qx, qw = ob.onebit_mx4_quantize(x * 2.0 ** ex), ob.onebit_mx4_quantize(w * 2.0 ** ew)
        a, b = (ob.onebit_mx4_dequantize(q).double() for q in (qx, qw))
        want = (a @ b.t()).float()
        assert float(want[0, 0]) == (2.0 ** (ex + ew - 2) if ex + ew < 130 else float("inf"))
        assert torch.equal(want[:, 1], -want[:, 0]) and (want[:, 2:] == 0).all()
        assert torch.equal(ob.onebit_mx4_matmul(qx, qw, dtype=F32), want)
        assert torch.equal(ob.onebit_mx4_linear(x * 2.0 ** ex, qw), want)
        assert torch.equal(ob.onebit_mx4_matmul(qx, qw), want.bfloat16())
