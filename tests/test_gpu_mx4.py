"""Matrices in microscaled 4-bit floating point on the GPU against the 64-bit reference.

Quantising and reading back are exact. A product's tolerance: an instruction adds 64 exact products
to the sum; whatever its order, no term passes through more than 7 roundings there and 7 more when
parts are joined, each at most 2^-23 of the sum of magnitudes (2^-24 to nearest, twice that where a
term is cut off). With bf16 results, half a step of the result (2^-8 of it) is added.
"""
import itertools

import numpy as np
import pytest
import torch

import communication_compressed_optimizer_momentum_b200 as ob
import mx4_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def matrix(rows, cols, dtype=F32, seed=0):
    """Normal values whose blocks differ in size by up to 2^16 either way, zeros among them."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, cols, device=DEV, generator=gen)
    x *= torch.exp2(torch.randint(-16, 17, (rows, cols // 16 + 1), device=DEV, generator=gen)
                    .repeat_interleave(16, 1)[:, :cols])
    x[torch.rand(rows, cols, device=DEV, generator=gen) < 0.05] = 0
    return x.to(dtype)


def check(q, x, seed=None):
    """An Mx4 against the reference's bytes for the matrix x; returns the values."""
    code, e = ref.quantize(x.float().cpu().numpy(), seed)
    packed, scales = ref.pack(code, e)
    assert q.shape == tuple(x.shape)
    assert np.array_equal(q.scales.cpu().numpy().ravel()[:scales.size], scales)
    assert np.array_equal(q.codes.cpu().numpy().reshape(packed.shape), packed)
    return ref.values(code, e, x.shape[1])


SIZES = [(1, 1), (1, 32), (1, 33), (31, 32), (32, 31), (33, 65), (128, 128), (129, 127), (127, 257),
         (5, 2000), (2000, 5), (300, 513), (640, 1024)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_and_back(rows, cols, rounding, dtype):
    x = matrix(rows, cols, dtype, rows + cols)
    seed = 12345678901234567
    at = (seed, seed + 1) if rounding == "stochastic" else (None, None)
    kw = dict(rounding=rounding, seed=seed)
    q, t = ob.onebit_mx4_quantize(x, forms="both", **kw)
    values = [check(q, x, at[0]), check(t, x.t(), at[1])]
    check(ob.onebit_mx4_quantize(x, **kw), x, at[0])
    check(ob.onebit_mx4_quantize(x, forms="columns", **kw), x.t(), at[1])
    for m, v in zip((q, t), values):
        assert np.array_equal(ob.onebit_mx4_dequantize(m).cpu().numpy(), v)
        assert np.array_equal(ob.onebit_mx4_dequantize(m, dtype=BF16).float().cpu().numpy(), v)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_values_at_borders(dtype):
    """Ties, zeros of both signs, the smallest and largest values, infinities and NaN."""
    tiny, big = 2.0 ** -126, 2.0 ** 127
    blocks = [
        [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 0.0, -0.0],
        [6.03125, 1, 2, 3], [7.9375, 3.96875], [4, 0.2490234375, 0.251953125], [0.0] * 32, [-0.0] * 32,
        [tiny], [tiny / 4, tiny / 64, -tiny / 128], [6 * tiny, tiny, tiny / 2], [2 * tiny, tiny],
        [1.5 * big, big, 2.0 ** 100, 1], [-1.5 * big, tiny], [1.5078125 * big, 1], [float("inf"), 1],
        [1, float("-inf")], [float("nan"), 5], [1, 2, float("nan")],
    ]
    x = torch.zeros(2, len(blocks) * 32, dtype=torch.float64)
    for i, b in enumerate(blocks):
        x[0, i * 32:i * 32 + len(b)] = torch.tensor(b, dtype=torch.float64)
        x[1, i * 32 + 32 - len(b):i * 32 + 32] = -torch.tensor(b, dtype=torch.float64)
    x = x.to(dtype).to(DEV)
    for seed in (None, 3):
        kw = dict(rounding="nearest" if seed is None else "stochastic", seed=3)
        q = ob.onebit_mx4_quantize(x, **kw)
        v = check(q, x, seed)
        t = ob.onebit_mx4_quantize(x.t().contiguous(), forms="columns", **{**kw, "seed": 2})
        check(t, x, seed)
        for out in (F32, BF16):
            got = ob.onebit_mx4_dequantize(q, dtype=out).double().cpu().numpy()
            assert np.array_equal(got, v, equal_nan=True)
            assert np.array_equal(np.isnan(got[0]).reshape(-1, 32).all(1),
                                  np.arange(len(blocks)) >= 12)


def test_stochastic_rounding_is_unbiased():
    """The mean of 4096 roundings is the value, within five standard deviations and the 2^-17 of a
    step that 16 bits lose."""
    n = 4096
    row = torch.linspace(-6, 6, 32, device=DEV)
    x = row.repeat(n, 1)
    v = ob.onebit_mx4_dequantize(ob.onebit_mx4_quantize(x, rounding="stochastic", seed=9)).double()
    a = row.abs().double()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    assert ((v.mean(0) - row.double()).abs() <= 5 * step / 2 / n ** 0.5 + step * 2 ** -17).all()
    assert ((v - row.double()).abs() < step).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("start,extra", [(0, 8), (1, 8), (3, 3), (8, 16), (0, 1)])
@pytest.mark.parametrize("forms", ["rows", "both"])
def test_row_strides_and_addresses(dtype, start, extra, forms):
    wide = matrix(70, 200 + extra + start, dtype, 4)
    x = wide[:, start:start + 200]
    q = ob.onebit_mx4_quantize(x, forms=forms)
    if forms == "both":
        check(q[1], x.t())
        q = q[0]
    v = check(q, x)
    out = torch.full((70, 200 + extra + start), 7.0, device=DEV, dtype=dtype)
    ob.onebit_mx4_dequantize(q, out=out[:, start:start + 200])
    assert np.array_equal(out[:, start:start + 200].float().cpu().numpy(), v)
    out[:, start:start + 200] = 7.0
    assert (out == 7.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (100, 320, 0), (33, 77, 5), (200, 130, 6)])
def test_error_feedback(rows, cols, pad, rounding, dtype):
    """Three messages in a row: each carries what the one before lost: to nearest exactly (a value
    that is not rounded to zero is between half and twice what it is held as, so that fp32 holds the
    difference), stochastically rounded once (a value far below what it is rounded up to is not)."""
    e = torch.zeros(rows, cols + pad, device=DEV)[:, :cols]
    held = np.zeros((rows, cols), dtype=np.float32)
    for step in range(3):
        x = matrix(rows, cols, dtype, step)
        q = ob.onebit_mx4_quantize(x, rounding=rounding, seed=step, residual=e)
        y = x.float().cpu().numpy() + held
        v = check(q, torch.from_numpy(y), step if rounding == "stochastic" else None)
        held = (y.astype(np.float64) - v).astype(np.float32)
        if rounding == "nearest":
            assert np.array_equal(held.astype(np.float64), y.astype(np.float64) - v)
        assert np.array_equal(e.cpu().numpy(), held)
    x[0, 0] = float("inf")
    ob.onebit_mx4_quantize(x, rounding=rounding, residual=e)
    assert e[0, :32].isnan().all() and not e[0, 32:].isnan().any()


def quantized(rows, cols, seed, big=4):
    """A matrix in 4 bits with blocks of different sizes, and its values in 64 bits."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, cols, device=DEV, generator=gen)
    x *= torch.exp2(torch.randint(-big, big + 1, (rows, cols // 32 + 1), device=DEV, generator=gen)
                    .repeat_interleave(32, 1)[:, :cols])
    q = ob.onebit_mx4_quantize(x)
    return q, ob.onebit_mx4_dequantize(q).double()


def tolerance(a, b, k):
    return (7 * -(-k // 64) + 7) * 2.0 ** -23 * (a.abs() @ b.abs().t())


PRODUCTS = [(2, 33, 31), (3, 129, 8193), (4, 6000, 1000), (4, 40, 20000), (4, 9000, 1500), (1, 1, 1), (1, 128, 64), (1, 129, 65), (16, 127, 256), (17, 1, 257), (32, 256, 128),
            (33, 100, 31), (64, 130, 1000), (65, 128, 2048), (100, 1000, 96), (128, 128, 512),
            (129, 300, 320), (256, 256, 256), (257, 129, 513), (300, 2000, 160), (1000, 77, 999),
            (1, 6400, 1600), (24, 5003, 1600), (2100, 2050, 700), (513, 50, 9000), (40, 40, 20000),
            # every width of tiles, split and not, with pairs whose second block has no columns, at
            # strides that TMA takes and others
            (12, 300, 5000), (9, 5003, 2100), (1000, 777, 1999), (1025, 1100, 9000), (5000, 3900, 600),
            (3000, 3900, 2000), (4100, 1001, 4000)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(m, n, k):
    (qa, a), (qb, b) = quantized(m, k, 1), quantized(n, k, 2)
    want, tol = a @ b.t(), tolerance(a, b, k)
    f = ob.onebit_mx4_matmul(qa, qb, dtype=F32)
    assert f.dtype == F32 and f.shape == (m, n)
    assert ((f.double() - want).abs() <= tol).all()
    h = ob.onebit_mx4_matmul(qa, qb)
    assert h.dtype == BF16
    assert ((h.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()
    base = torch.randn(m, n, device=DEV)
    acc = ob.onebit_mx4_matmul(qa, qb, out=base.clone(), accumulate=True)
    assert torch.equal(acc, base + f)                 # one addition of the same sums
    assert torch.equal(ob.onebit_mx4_matmul(qa, qb, dtype=F32), f)
    assert ob.onebit_mx4_status() == 0


@pytest.mark.parametrize("m,n,k", [(7, 300, 8192), (200, 200, 4096), (1500, 1111, 1024), (300, 5000, 192)])
def test_product_of_small_numbers_is_exact(m, n, k):
    """All products are multiples of 2^-4 and no sum of magnitudes reaches 2^20: nothing rounds."""
    (qa, a), (qb, b) = quantized(m, k, 3, big=0), quantized(n, k, 4, big=0)
    unit = 2.0 ** 6                                    # magnitudes below 6: scales 2^-2 to 2^0
    assert float((a * unit).frac().abs().max()) == 0 and float((b * unit).frac().abs().max()) == 0
    a, b = (x.clamp(-1.5, 1.5) for x in (a, b))
    qa, qb = (ob.onebit_mx4_quantize((x * 4).round().float() / 4) for x in (a, b))
    a, b = (ob.onebit_mx4_dequantize(q).double() for q in (qa, qb))
    assert float((a * 4).frac().abs().max()) == 0 and float((b * 4).frac().abs().max()) == 0
    assert float((a.abs() @ b.abs().t()).max()) < 2 ** 20
    assert torch.equal(ob.onebit_mx4_matmul(qa, qb, dtype=F32).double(), a @ b.t())


@pytest.mark.parametrize("m,n,k", [(5, 300, 1000), (3, 70, 500), (150, 140, 3000), (260, 40000, 64)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_product_into_a_slice(m, n, k, dtype):
    (qa, a), (qb, b) = quantized(m, k, 5), quantized(n, k, 6)
    want = ob.onebit_mx4_matmul(qa, qb, dtype=dtype)
    room = torch.full((m + 2, n + 5), 3.0, device=DEV, dtype=dtype)
    out = room[1:-1, 2:-3]
    assert ob.onebit_mx4_matmul(qa, qb, out=out) is out
    assert torch.equal(out, want)
    out.fill_(3.0)
    assert (room == 3.0).all()


def test_product_with_nan_blocks():
    """A NaN block reaches its row or column and nothing else."""
    for m, n, k in ((3, 300, 700), (5, 300, 700), (300, 200, 4000)):
        x, y = matrix(m, k, seed=1) * 2.0 ** -8, matrix(n, k, seed=2) * 2.0 ** -8
        x[m // 2, k - 1] = float("nan")
        y[n - 1, 0] = float("inf")
        qa, qb = ob.onebit_mx4_quantize(x), ob.onebit_mx4_quantize(y)
        a, b = (ob.onebit_mx4_dequantize(q).double() for q in (qa, qb))
        got = ob.onebit_mx4_matmul(qa, qb, dtype=F32).double()
        nan = torch.zeros(m, n, dtype=torch.bool, device=DEV)
        nan[m // 2], nan[:, n - 1] = True, True
        assert torch.equal(got.isnan(), nan)
        a, b = a.nan_to_num(0.0), b.nan_to_num(0.0)
        assert ((got - a @ b.t()).abs() <= tolerance(a, b, k))[~nan].all()


def test_extreme_scales():
    """Exponents at both ends: products are right wherever fp32 holds them."""
    for (ea, eb), m in itertools.product(((-126, 100), (120, -120), (-60, -60), (60, 60), (-126, 0),
                                          (125, -10)), (3, 20)):
        x = matrix(m, 256, seed=3).clamp(-1, 1) * 2.0 ** ea
        y = matrix(140, 256, seed=4).clamp(-1, 1) * 2.0 ** eb
        qa, qb = ob.onebit_mx4_quantize(x), ob.onebit_mx4_quantize(y)
        a, b = (ob.onebit_mx4_dequantize(q).double() for q in (qa, qb))
        got, want = ob.onebit_mx4_matmul(qa, qb, dtype=F32).double(), a @ b.t()
        # terms below the smallest normal value may count as zero
        assert ((got - want).abs() <= tolerance(a, b, 256) + 256 * 2.0 ** -126).all(), (ea, eb)


def test_empty_and_one():
    for m, n, k in itertools.product((0, 1), repeat=3):
        qa = ob.onebit_mx4_quantize(torch.ones(m, k, device=DEV))
        qb = ob.onebit_mx4_quantize(torch.full((n, k), 3.0, device=DEV))
        for dtype in (F32, BF16):
            out = ob.onebit_mx4_matmul(qa, qb, dtype=dtype)
            assert out.shape == (m, n) and (out == 3.0 * k).all()
        acc = ob.onebit_mx4_matmul(qa, qb, out=torch.ones(m, n, device=DEV), accumulate=True)
        assert (acc == 1 + 3.0 * k).all()
        assert ob.onebit_mx4_dequantize(qa).shape == (m, k)
        both = ob.onebit_mx4_quantize(torch.ones(m, k, device=DEV), forms="both")
        assert both[1].shape == (k, m)
    wide = torch.full((4, 9), 2.0, device=DEV)
    q = ob.onebit_mx4_quantize(torch.ones(4, 0, device=DEV)), ob.onebit_mx4_quantize(
        torch.ones(5, 0, device=DEV))
    ob.onebit_mx4_matmul(*q, out=wide[:, 2:7])
    assert (wide[:, 2:7] == 0).all() and (wide[:, :2] == 2).all() and (wide[:, 7:] == 2).all()


@pytest.mark.parametrize("case", ["quantize", "product"])
def test_more_than_2_to_the_31_elements(case):
    """Places beyond 32 bits: the last rows against the reference."""
    if case == "quantize":
        rows, cols = 70_000, 40_000
        x = torch.empty(rows, cols, dtype=BF16, device=DEV)
        x.normal_(generator=torch.Generator(device=DEV).manual_seed(1))
        q, t = ob.onebit_mx4_quantize(x, forms="both", rounding="stochastic", seed=5)
        for rows_of, at, seed in ((x, rows - 3, 5), (x.t(), cols - 3, 6)):
            m = (q, t)[seed - 5]
            want = rows_of[at:].float().cpu().numpy()
            code, e = ref.quantize(want, seed, row0=at)
            packed, _ = ref.pack(code, e)
            assert np.array_equal(m.codes[at:].cpu().numpy(), packed)
            got = torch.empty(m.rows, m.cols, dtype=BF16, device=DEV)
            ob.onebit_mx4_dequantize(m, out=got)
            assert np.array_equal(got[at:].float().cpu().numpy(), ref.values(code, e, m.cols))
            del got
        return
    m, n, k = 50_000, 50_000, 70
    (qa, a), (qb, b) = quantized(m, k, 1), quantized(n, k, 2)
    out = ob.onebit_mx4_matmul(qa, qb)
    for rows in (slice(0, 3), slice(m - 3, m)):
        want, tol = a[rows] @ b.t(), tolerance(a[rows], b, k)
        assert ((out[rows].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()


def test_another_stream_and_captured_calls():
    x = matrix(300, 500, seed=1)
    w = ob.onebit_mx4_quantize(matrix(200, 500, seed=2))
    want = ob.onebit_mx4_matmul(ob.onebit_mx4_quantize(x), w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        q = ob.onebit_mx4_quantize(x, stream=stream)
        got = ob.onebit_mx4_matmul(q, w, stream=stream)
        back = ob.onebit_mx4_dequantize(q, stream=stream)
        del q
        side.synchronize()
        assert torch.equal(got, want) and back.shape == x.shape
    # captured: a replay takes the values that are there then; two graphs share nothing
    buf, out, out2 = torch.zeros_like(x), torch.empty_like(want), torch.empty_like(want)
    q, q2 = ob.Mx4.empty(300, 500), ob.Mx4.empty(300, 500)
    graphs = []
    for qq, o in ((q, out), (q2, out2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ob.onebit_mx4_quantize(buf, out=qq)
            ob.onebit_mx4_matmul(qq, w, out=o)
        graphs.append(g)
    buf.copy_(x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(out2, want)


def test_captured_with_a_fork_and_other_nodes_between():
    """Launches that may begin early, after a join of two streams, a copy and a fill."""
    x = matrix(300, 500, seed=1)
    w = ob.onebit_mx4_quantize(matrix(200, 500, seed=2))
    want = ob.onebit_mx4_matmul(ob.onebit_mx4_quantize(x), w)
    buf, out, out2 = torch.zeros_like(x), torch.ones_like(want), torch.ones(300, 200, device=DEV)
    q, q2 = ob.Mx4.empty(300, 500), ob.Mx4.empty(300, 500)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        buf.copy_(x)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            ob.onebit_mx4_quantize(buf, out=q)
        ob.onebit_mx4_quantize(buf, out=q2)
        here.wait_stream(side)
        ob.onebit_mx4_matmul(q, w, out=out)
        out2.zero_()
        ob.onebit_mx4_matmul(q2, w, out=out2, accumulate=True)
    for _ in range(3):
        buf.fill_(float("nan"))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out2.bfloat16(), want)


def test_products_on_two_streams_at_once():
    """Both fill the GPU, with pairs and with clusters of other sizes."""
    shapes = [(1024, 2048, 2048), (16, 2048, 8192), (300, 4000, 1000), (4, 4096, 1024), (30, 100, 16384)]
    data = [(quantized(m, k, 1)[0], quantized(n, k, 2)[0]) for m, n, k in shapes]
    want = [ob.onebit_mx4_matmul(a, b, dtype=F32) for a, b in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                for a, b in data[::1 if i else -1]:
                    got[i].append(ob.onebit_mx4_matmul(a, b, dtype=F32))
    torch.cuda.synchronize()
    for i in range(2):
        for j, x in enumerate(got[i]):
            k = j % len(data)
            assert torch.equal(x, want[k if i else len(data) - 1 - k])
    assert ob.onebit_mx4_status() == 0


def test_a_chain_of_short_calls():
    """Each reads what the one before wrote, many times over: none starts too early. (The values are
    brought back to 1 at most; they would grow to infinity.)"""
    w = ob.Mx4Linear(torch.randn(64, 64, device=DEV) * 0.2)
    x = torch.randn(130, 64, device=DEV)
    y, z = x.clone(), x
    for i in range(200):
        y = ob.onebit_mx4_dequantize(ob.onebit_mx4_quantize(w.forward(y) + x, forms="rows"))
        y = y / y.abs().amax()
    for i in range(200):
        torch.cuda.synchronize()
        z = w.forward(z)
        torch.cuda.synchronize()
        q = ob.onebit_mx4_quantize(z + x)
        torch.cuda.synchronize()
        z = ob.onebit_mx4_dequantize(q)
        z = z / z.abs().amax()
    assert torch.equal(y, z) and z.isfinite().all()


def test_refusals_on_the_gpu():
    x = torch.zeros(4, 64, device=DEV)
    q = ob.onebit_mx4_quantize(x)
    for bad, error in ((x.double(), TypeError), (x.half(), TypeError), (x.t(), ValueError),
                       (x.view(-1), ValueError), (x[:, ::2], ValueError)):
        with pytest.raises(error):
            ob.onebit_mx4_quantize(bad)
    with pytest.raises(ob.OneBitError, match="stride"):
        ob.onebit_mx4_quantize(torch.zeros(64, device=DEV).expand(4, 64))
    with pytest.raises(ValueError, match="size"):
        ob.onebit_mx4_quantize(x, out=ob.Mx4.empty(4, 65))
    with pytest.raises(ValueError, match="size"):
        ob.onebit_mx4_quantize(x, residual=x[:3])
    with pytest.raises(TypeError):
        ob.onebit_mx4_quantize(x, residual=x.bfloat16())
    with pytest.raises(ob.OneBitError, match="overlaps"):
        ob.onebit_mx4_quantize(x, residual=x)
    with pytest.raises(ValueError, match="needs at least"):
        ob.onebit_mx4_dequantize(ob.Mx4(q.codes, q.scales[:100], 4, 64))
    with pytest.raises(ValueError, match="needs at least"):
        ob.onebit_mx4_dequantize(ob.Mx4(q.codes, q.scales, 5, 64))
    with pytest.raises(TypeError):
        ob.onebit_mx4_dequantize(q, dtype=torch.float16)
    with pytest.raises(ValueError, match="columns"):
        ob.onebit_mx4_matmul(q, ob.onebit_mx4_quantize(x[:, :63]))
    with pytest.raises(ValueError, match="accumulate"):
        ob.onebit_mx4_matmul(q, q, accumulate=True)
    with pytest.raises(ob.OneBitError, match="float32 out"):
        ob.onebit_mx4_matmul(q, q, out=torch.zeros(4, 4, device=DEV, dtype=BF16), accumulate=True)
    with pytest.raises(ValueError, match="size"):
        ob.onebit_mx4_matmul(q, q, out=torch.zeros(4, 5, device=DEV))
    with pytest.raises(TypeError):
        ob.onebit_mx4_matmul(q, q, out=torch.zeros(4, 4, device=DEV), dtype=BF16)
    moved = torch.zeros(q.codes.numel() + 16, dtype=torch.uint8, device=DEV)[8:8 + q.codes.numel()]
    with pytest.raises(ob.OneBitError, match="aligned"):
        ob.onebit_mx4_dequantize(ob.Mx4(moved, q.scales, 4, 64))


# ----------------------------------------------------------------------------------------------
# the linear layer

def values(q):
    return ob.onebit_mx4_dequantize(q).double()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,inner,outer", [((1,), 64, 96), ((4,), 2000, 5000), ((2, 2), 77, 33),
                                                ((), 64, 40), ((3, 50), 200, 130), ((515,), 96, 1000)])
def test_linear_passes(tokens, inner, outer, dtype):
    w = torch.randn(outer, inner, device=DEV) * 0.1
    x = torch.randn(*tokens, inner, device=DEV).to(dtype)
    dy = torch.randn(*tokens, outer, device=DEV).to(dtype)
    flat, dflat = x.view(-1, inner), dy.view(-1, outer)
    t = flat.shape[0]
    linear = ob.Mx4Linear(w)
    y, kept = linear.forward(x, keep=True)
    assert torch.equal(y, linear.forward(x)) and y.shape == (*tokens, outer) and y.dtype == dtype
    dx, dw = linear.backward(dy, kept, seed=4)
    assert dx.shape == x.shape and dx.dtype == dtype and dw.shape == w.shape and dw.dtype == F32

    def q(m, seed=None):
        m = m.float().cpu().numpy()
        return torch.from_numpy(ref.values(*ref.quantize(m, seed), m.shape[1])).to(DEV)

    for got, a, b, k in ((y, q(flat), q(w), inner), (dx, q(dflat, 4), q(w.t()), outer),
                         (dw, q(dflat.t(), 5), q(flat.t()), t)):
        want, tol = a @ b.t(), tolerance(a, b, k)
        if got.dtype == BF16:
            tol = tol + 2.0 ** -8 * (want.abs() + tol)
        assert ((got.view(want.shape).double() - want).abs() <= tol).all()
    # parts of the backward pass alone, and into a gradient
    assert torch.equal(linear.backward(dy, seed=4)[0], dx)
    only = linear.backward(dy, kept, seed=4, need_dx=False)
    assert only[0] is None and torch.equal(only[1], dw)
    grad = torch.ones_like(w)
    assert linear.backward(dy, kept, seed=4, grad=grad, accumulate=True)[1] is grad
    assert torch.equal(grad, 1 + dw)
    half = torch.empty(outer, inner, device=DEV, dtype=BF16)
    linear.backward(dy, kept, seed=4, grad=half)
    assert torch.equal(half, dw.bfloat16())


def test_linear_gradients_against_differences():
    """With values that 4 bits hold, the passes are the exact linear map and its gradients: the loss
    <dy, x W^T> changes by exactly <dx, d> and <dW, d>, in directions that are held too."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4], device=DEV)

    def held(rows, cols):      # every block along either axis holds a 6, so its exponent is 0
        v = table[torch.randint(0, 7, (rows, cols), device=DEV, generator=gen)]
        v = v * (torch.randint(0, 2, (rows, cols), device=DEV, generator=gen) * 2 - 1)
        r, c = torch.arange(rows, device=DEV)[:, None], torch.arange(cols, device=DEV)
        return torch.where((r + c) % 32 == 0, 6.0, v)

    t, inner, outer = 64, 96, 160
    x, w, dy = held(t, inner), held(outer, inner), held(t, outer)

    def loss(x, w):
        return float((dy.double() * ob.Mx4Linear(w).forward(x).double()).sum())

    linear = ob.Mx4Linear(w)
    _, kept = linear.forward(x, keep=True)
    dx, dw = linear.backward(dy, kept, seed=1)
    assert torch.equal(dx.double(), dy.double() @ w.double())
    assert torch.equal(dw.double(), dy.double().t() @ x.double())
    for i, j in ((1, 0), (5, 40), (63, 95)):
        for m, g, f in ((x, dx, lambda z: loss(z, w)), (w, dw, lambda z: loss(x, z))):
            z = m.clone()
            z[i, j] = 1.0 if z[i, j] != 1 and z[i, j] != 6 else 2.0
            if m[i, j] == 6:
                continue
            assert f(z) - f(m) == float(g[i, j].double() * (z[i, j] - m[i, j]).double())


@pytest.mark.parametrize("state,max_norm,ptype", [("f32", None, F32), ("q8", 1.0, F32), ("f32", 1.0, BF16)])
def test_training_with_adamw(state, max_norm, ptype):
    """Steps of a two-layer model: forward, backward and AdamW, which quantises the weights again; by
    calls and as one captured graph, with the same results bit for bit."""
    gen = torch.Generator(device=DEV).manual_seed(6)

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=gen)

    start = [(normal(96, 64) * 0.1).to(ptype), (normal(32, 96) * 0.1).to(ptype), normal(96).to(ptype)]
    x, target = normal(200, 64).bfloat16(), normal(200, 32).bfloat16()

    def build():
        ps = [p.clone() for p in start]
        layers = [ob.Mx4Linear(p) for p in ps[:2]]
        gs = [torch.zeros(p.shape, device=DEV) for p in ps]
        return ps, layers, gs, ob.AdamW(ps, max_norm=max_norm, state=state)

    def step(ps, layers, gs, opt):
        h, k0 = layers[0].forward(x, keep=True)
        a = torch.relu(h + ps[2].to(h.dtype))
        y, k1 = layers[1].forward(a, keep=True)
        dy = (y - target) / 200
        da, _ = layers[1].backward(dy, k1, seed=1, grad=gs[1])
        dh = torch.where(a > 0, da, torch.zeros_like(da))
        layers[0].backward(dh, k0, seed=2, grad=gs[0], need_dx=False)
        torch.sum(dh.float(), 0, out=gs[2])
        opt.step(ps, gs, 1e-3, mx4=layers + [None])

    eager = build()
    for _ in range(4):
        step(*eager)
    graphed = build()
    step(*graphed)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*graphed)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert eager[3].counts() == graphed[3].counts() == (4, 0)
    for a, b in zip(eager[0] + eager[2], graphed[0] + graphed[2]):
        assert torch.equal(a, b) and a.isfinite().all()
    for p, layer in zip(eager[0], eager[1]):
        fresh = ob.Mx4Linear(p)
        for q, r in ((layer.w, fresh.w), (layer.wt, fresh.wt)):
            assert torch.equal(q.codes, r.codes) and torch.equal(q.scales, r.scales)
    assert not torch.equal(eager[0][0], start[0])


def test_linear_refusals():
    w = torch.randn(40, 64, device=DEV)
    linear, forward_only = ob.Mx4Linear(w), ob.Mx4Linear(w, backward=False)
    x, dy = torch.randn(5, 64, device=DEV), torch.randn(5, 40, device=DEV)
    y, kept = linear.forward(x, keep=True)
    assert torch.equal(forward_only.forward(x), y)
    assert linear.forward(x[:0]).shape == (0, 40)
    _, none = linear.forward(x[:0], keep=True)
    dx, dw = linear.backward(dy[:0], none)
    assert dx.shape == (0, 64) and (dw == 0).all()
    with pytest.raises(ValueError, match="columns"):
        linear.forward(dy)
    with pytest.raises(ValueError, match="columns"):
        linear.backward(x, kept)
    with pytest.raises(ValueError, match="kept"):
        linear.backward(dy[:4], kept)
    with pytest.raises(TypeError, match="Mx4"):
        linear.backward(dy, x)
    with pytest.raises(ValueError, match="kept"):
        linear.backward(dy, grad=w)
    with pytest.raises(ValueError, match="grad"):
        linear.backward(dy, kept, accumulate=True)
    with pytest.raises(ValueError, match="contiguous"):
        linear.forward(torch.zeros(3, 5, 128, device=DEV)[..., :64])
    with pytest.raises(TypeError):
        linear.forward(x.half())
    assert torch.equal(linear.forward(torch.cat([x, x], 1)[:, :64]), y)   # rows apart
    with pytest.raises(ValueError, match="backward=True"):
        forward_only.backward(dy)
    assert forward_only.backward(dy, kept, need_dx=False)[1].shape == (40, 64)
    with pytest.raises(ValueError, match="40 x 64"):
        linear.update(w.t())
    with pytest.raises(ValueError, match="cuda"):
        linear.update(w.cpu())
    opt = ob.AdamW([w, dy])
    before = w.clone()
    for mx4, error in (([linear], ValueError), ([None, linear], ValueError), ([w, None], TypeError)):
        with pytest.raises(error):
            opt.step([w, dy], [w.clone(), dy.clone()], 1e-3, mx4=mx4)
    assert torch.equal(w, before) and opt.counts() == (0, 0)
