"""AdamW over a list of tensors on the GPU, against the 64-bit implementation in
adamw_reference.py: every type, sizes from none to odd ones and to more than 2^31 elements, views at
odd addresses, short and long lists, what a call must leave as it is, non-finite values, streams and
graphs, and the operators in a row."""
import math

import numpy as np
import pytest
import torch

import communication_compressed_optimizer_momentum_b200 as ob
import adamw_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BLOCK = 256
HP = dict(lr=3e-3, beta1=0.9, beta2=0.999, eps=1e-8)
SHORT = [0, 1, 255, 256, 257, 4099, 0, 8, 70001, 2048]
LONG = [1 + (37 * i) % 700 for i in range(130)]
LONGER = [(i * 7919) % 900 for i in range(1700)]      # three launches
FILL = 77.0


def host(t):
    return t.detach().double().cpu().numpy()


class Problem:
    """Tensors as views of arenas (gaps between them hold FILL), and flat states whose places
    behind a tensor hold FILL too."""

    def __init__(self, sizes, ptype, gtype, align=16, seed=0, copies=False, eight=False,
                 sigma=1e-2, sparse=False):
        rng = np.random.default_rng(seed)
        self.sizes = sizes
        self.eight = eight
        self.hp = dict(HP)
        self.offsets, self.total = ob.onebit_adamw_layout(sizes)
        self.at = []
        n = 3 if align == 1 else 0                    # odd addresses, not only odd distances
        for s in sizes:
            self.at.append(n)
            n += -(-(s + 1) // align) * align
        self.room = n

        def arena(dtype, values):
            a = torch.full((self.room,), FILL, dtype=dtype, device=DEV)
            views = [a[i:i + s] for i, s in zip(self.at, sizes)]
            for view, x in zip(views, values):
                view.copy_(torch.from_numpy(x))
            return a, views
        per = [rng.standard_normal(s).astype(np.float32) for s in sizes]
        self.p_arena, self.p = arena(ptype, [x * 0.05 for x in per])
        grads = [(rng.standard_normal(s) * sigma).astype(np.float32) for s in sizes]
        if sparse:
            for x in grads:
                x[rng.random(x.size) < 0.3] = 0.0
        self.g_arena, self.g = arena(gtype, grads)
        self.c_arena, self.c = None, None
        if copies:
            self.c_arena, self.c = arena(torch.bfloat16, [x * 0 for x in per])
        inside = np.zeros(self.total, bool)
        for o, s in zip(self.offsets, sizes):
            inside[o:o + s] = True
        self.inside = inside
        m = np.where(inside, rng.standard_normal(self.total) * 0.3 * sigma, FILL)
        v = np.where(inside, rng.random(self.total) * sigma ** 2, FILL)
        if eight:
            # every code, the places behind a tensor too; exponents of the gradients' size
            def codes():
                return torch.from_numpy(rng.integers(0, 256, self.total).astype(np.uint8)).to(DEV)
            blocks = self.total // BLOCK
            km = rng.integers(115, 122, blocks).astype(np.uint8)
            kv = rng.integers(108, 118, blocks).astype(np.uint8)
            self.state = [codes(), codes(), torch.from_numpy(km).to(DEV),
                          torch.from_numpy(kv).to(DEV)]
        else:
            self.state = [torch.from_numpy(x.astype(np.float32)).to(DEV) for x in (m, v)]
        self.ctl = torch.zeros(8, dtype=torch.int64, device=DEV)
        self.wd = [0.1 if s > 300 else 0.0 for s in sizes]

    def moments64(self):
        if not self.eight:
            return [host(x) for x in self.state]
        c = [x.cpu().numpy() for x in self.state]
        return ref.decode64(c[0], c[2], True), ref.decode64(c[1], c[3], False)

    def set_t(self, t, b1=0.9, b2=0.999):
        self.ctl[0] = t
        self.ctl[2:4] = torch.tensor([1 - b1 ** t, 1 - b2 ** t], dtype=torch.float64,
                                     device=DEV).view(torch.int64)

    def step(self, lr=None, scale=None, seed=5, bias=True, stream=None, grads=None):
        lr = HP["lr"] if lr is None else lr
        kw = dict(copies=self.c, grad_scale=scale, bias_correction=bias, stream=stream)
        args = (self.ctl, lr, self.hp["beta1"], self.hp["beta2"], self.hp["eps"], self.wd)
        grads = self.g if grads is None else grads
        if self.eight:
            ob.onebit_adamw8_step(self.p, grads, *self.state, *args, seed=seed, **kw)
        else:
            ob.onebit_adamw_step(self.p, grads, *self.state, *args, **kw)

    def everything(self):
        return [x.clone() for x in [self.p_arena, *self.state, self.ctl[:4]]
                + ([self.c_arena] if self.c else [])]


def same_bits(a, b):
    return all(torch.equal(x.reshape(-1).view(torch.uint8), y.reshape(-1).view(torch.uint8))
               for x, y in zip(a, b))


def check_step(pr, scale, t, seed=5, bias=True):
    """Run step t of a problem and check everything it writes and leaves."""
    p0, g0 = [host(x) for x in pr.p], [host(x) for x in pr.g]
    m0, v0 = pr.moments64()
    before = [x.cpu().numpy().copy() for x in pr.state]
    s = None if scale is None else torch.tensor([scale], dtype=torch.float32, device=DEV)
    s64 = 1.0 if scale is None else float(np.float32(scale))
    pr.set_t(t - 1, pr.hp["beta1"], pr.hp["beta2"])
    pr.step(scale=s, seed=seed, bias=bias)
    torch.cuda.synchronize()
    assert pr.ctl[:2].tolist() == [t, 0]
    after = [x.cpu().numpy() for x in pr.state]
    # the gaps and the places behind the tensors
    p_arena = host(pr.p_arena)
    gaps = np.ones(pr.room, bool)
    for a, n in zip(pr.at, pr.sizes):
        gaps[a:a + n] = False
    assert (p_arena[gaps] == FILL).all()
    if pr.c:
        assert (host(pr.c_arena)[gaps] == FILL).all()
    for x, y in zip(before[:2], after[:2]):
        assert np.array_equal(x[~pr.inside], y[~pr.inside])
    ptype = pr.p_arena.dtype
    for i, n in enumerate(pr.sizes):
        if n == 0:
            continue
        o = slice(pr.offsets[i], pr.offsets[i] + n)
        (p1, m1, v1), (ep, em, ev) = ref.step64(
            p0[i], g0[i], m0[o], v0[o], t, HP["lr"], pr.hp["beta1"], pr.hp["beta2"], pr.hp["eps"],
            pr.wd[i], s64, bias)
        got = host(pr.p[i])
        bound = ep if ptype == torch.float32 else ref.bf16_bound(p1, ep)
        assert (np.abs(got - p1) <= bound).all(), (i, n, np.max(np.abs(got - p1) / bound))
        if pr.c:
            assert torch.equal(pr.c[i], pr.p[i].to(torch.bfloat16))
        if not pr.eight:
            assert (np.abs(after[0][o] - m1) <= em).all(), (i, n)
            assert (np.abs(after[1][o] - v1) <= ev).all(), (i, n)
            continue
        # 8 bits: the exact code that the documented rounding of the fp32 moments gives
        m32, v32 = ref.moments32(g0[i], m0[o], v0[o], pr.hp["beta1"], pr.hp["beta2"], s64)
        blocks = -(-n // BLOCK)
        words = ref.random_words(np.arange(o.start, o.start + blocks * BLOCK), seed, t)
        for x, x64, e64, codes, exps, signed, r in (
                (m32, m1, em, after[0], after[2], True, words >> 16),
                (v32, v1, ev, after[1], after[3], False, words & 0xFFFF)):
            padded = np.zeros(blocks * BLOCK)
            padded[:n] = x
            want, k = ref.encode64(padded, signed, r / 65536)
            b = slice(o.start // BLOCK, o.start // BLOCK + blocks)
            assert np.array_equal(exps[b], k), (i, n, signed)
            assert np.array_equal(codes[o], want[:n]), (i, n, signed)
            # and within one step of the 64-bit value: 1/8 of its binade, or the smallest step
            full = np.zeros(blocks * BLOCK, np.uint8)
            full[:n] = codes[o]
            held = ref.decode64(full, exps[b], signed)[:n]
            top = 15 if signed else 31
            least = np.repeat(np.ldexp(1.0, exps[b].astype(int) - 127 - top + 1 - 3), BLOCK)[:n]
            binade = np.ldexp(1.0, np.frexp(np.abs(x64) + e64)[1] - 4)
            assert (np.abs(held - x64) <= np.maximum(binade, least) + e64).all(), (i, n, signed)


TYPES = [(torch.float32, torch.float32, False), (torch.float32, torch.bfloat16, True),
         (torch.bfloat16, torch.bfloat16, False), (torch.bfloat16, torch.float32, False)]
IDS = ["f32_f32", "f32_bf16_copy", "bf16_bf16", "bf16_f32"]


@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
@pytest.mark.parametrize("align", [1, 8, 16])
@pytest.mark.parametrize("ptype,gtype,copies", TYPES, ids=IDS)
def test_step(ptype, gtype, copies, align, eight):
    pr = Problem(SHORT, ptype, gtype, align, seed=align, copies=copies, eight=eight, sparse=True)
    check_step(pr, 0.37, 1)
    check_step(pr, None, 2)
    check_step(pr, 1.0, 1000, seed=(1 << 40) + 9)


@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
@pytest.mark.parametrize("sizes", [LONG, LONGER], ids=["130", "1700"])
def test_step_over_long_lists(sizes, eight):
    pr = Problem(sizes, torch.float32, torch.float32, 1, seed=3, eight=eight)
    check_step(pr, 0.5, 7)


@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
@pytest.mark.parametrize("first", [1, 300, 600, 800])
def test_second_launch_begins_anywhere_in_a_unit(first, eight):
    """More than 800 tensors take two launches; the second one's first block falls on each place
    among the four blocks that a warp takes at a time, with large aligned tensors behind it."""
    pr = Problem([first] + [100] * 802 + [5000, 70_001, 4096], torch.float32, torch.float32, 16,
                 seed=first, eight=eight)
    check_step(pr, 0.5, 3)


@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
def test_step_without_elements_counts(eight):
    pr = Problem([0, 0], torch.float32, torch.float32, eight=eight)
    check_step(pr, 0.5, 3)
    empty = Problem([], torch.float32, torch.float32, eight=eight)
    empty.step()
    assert empty.ctl[:2].tolist() == [1, 0]


@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
def test_address_does_not_matter(eight):
    """The same values at 16-byte and at odd addresses: the same bits."""
    a = Problem(SHORT, torch.float32, torch.float32, 16, seed=4, copies=True, eight=eight)
    b = Problem(SHORT, torch.float32, torch.float32, 1, seed=4, copies=True, eight=eight)
    for _ in range(3):
        a.step()
        b.step()
    assert same_bits(a.state + a.p + a.c + [a.ctl[:4]], b.state + b.p + b.c + [b.ctl[:4]])


@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
@pytest.mark.parametrize("beta1,beta2,eps", [
    (0.0, 0.999, 1e-8), (0.9, 0.0, 1e-8), (0.0, 0.0, 1e-3), (0.95, 0.9999, 1e-6),
    (0.9, 0.999, 1e-14), (1e-30, 0.999, 1e-8), (0.9, 0.999, 1e25)])
def test_other_hyperparameters(beta1, beta2, eps, eight):
    """Betas of 0 and next to it, and an eps that is too small or too large for the 8-bit step's
    approximations: the plain form."""
    pr = Problem(SHORT, torch.float32, torch.bfloat16, 16, seed=12, eight=eight)
    pr.hp.update(beta1=beta1, beta2=beta2, eps=eps)
    check_step(pr, 0.8, 1)
    check_step(pr, None, 2)


def test_bias_correction_off_and_decay_off():
    pr = Problem(SHORT, torch.float32, torch.float32, seed=6)
    pr.wd = [0.0] * len(SHORT)
    check_step(pr, None, 5, bias=False)


@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
def test_equals_the_warmup_step_and_hands_over_to_one_bit_adam(gdtype):
    """Without bias correction and decay, and with betas that are fp32 values, a step is the
    library's own Adam warm-up with one worker, bit for bit; a run begun here continues there."""
    d, C = 10_001, 4096
    b1, b2 = float(np.float32(0.9)), float(np.float32(0.999))
    gen = torch.Generator(device=DEV).manual_seed(1)
    xa = torch.randn(d, device=DEV, generator=gen) * 0.05
    xb = xa.clone()
    one = ob.OneBitAdam(d, 1, C, b1, b2, 1e-8, grad_dtype=gdtype, device=DEV)
    two = ob.OneBitAdam(d, 1, C, b1, b2, 1e-8, grad_dtype=gdtype, device=DEV)
    cuts = [0, 17, 300, 5000, d]
    views = [xb[i:j] for i, j in zip(cuts, cuts[1:])]
    opt = ob.AdamW(views, b1, b2, 1e-8, weight_decay=0.0, bias_correction=False)
    grads = [(torch.randn(d, device=DEV, generator=gen) * 1e-2).to(gdtype) for _ in range(6)]
    for g in grads[:3]:
        one.warmup_step(xa, g.view(1, d), 1e-3)
        opt.step(views, [g[i:j] for i, j in zip(cuts, cuts[1:])], 1e-3)
    m, v = opt.get_state()
    flat = [torch.cat([x[o:o + n] for o, n in zip(opt.offsets, opt.lengths)]) for x in (m, v)]
    assert same_bits([xa, one.get_state("m"), one.get_state("v")], [xb, *flat])
    two.set_state("m", flat[0])
    two.set_state("v", flat[1])
    one.freeze()
    two.freeze()
    for g in grads[3:]:
        one.step(xa, g.view(1, d), 1e-3)
        two.step(xb, g.view(1, d), 1e-3)
    assert same_bits([xa], [xb])
    one.close()
    two.close()


@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan])
def test_a_scale_that_is_not_finite_leaves_the_step_out(eight, scale):
    pr = Problem(LONGER if scale == math.inf else SHORT, torch.float32, torch.bfloat16, 1,
                 copies=True, eight=eight)
    pr.set_t(4)
    before = pr.everything()
    pr.step(scale=torch.tensor([scale], device=DEV))
    assert pr.ctl[:2].tolist() == [4, 1]
    pr.ctl[1] = 0
    assert same_bits(before, pr.everything())
    check_step(pr, 0.5, 5)


@pytest.mark.parametrize("align", [1, 16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_bad_gradients_32(bad, align):
    """One element's gradient is not finite: that element's moments and parameter are not either,
    every other one is as if nothing had happened."""
    a = Problem([2500, 500], torch.float32, torch.float32, align, seed=2)
    b = Problem([2500, 500], torch.float32, torch.float32, align, seed=2)
    a.g[0][777] = bad
    a.step()
    b.step()
    assert not torch.isfinite(a.p[0][777]) and not torch.isfinite(a.state[0][777])
    a.p[0][777], a.state[0][777], a.state[1][777] = b.p[0][777], b.state[0][777], b.state[1][777]
    assert same_bits(a.everything(), b.everything())


@pytest.mark.parametrize("align", [1, 16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_bad_gradients_8(bad, align):
    """With 8-bit states the element's whole block of m and v reads as NaN afterwards; the
    parameters of this step and every other block are as if nothing had happened."""
    a = Problem([2500, 500], torch.float32, torch.float32, align, seed=2, eight=True)
    b = Problem([2500, 500], torch.float32, torch.float32, align, seed=2, eight=True)
    for i in (777, 2499):                          # in a whole block and in the last one
        a.g[0][i] = bad
    a.step()
    b.step()
    m, v = ob.onebit_adamw8_get_state(*a.state)
    hit = torch.zeros(a.total, dtype=torch.bool, device=DEV)
    hit[768:1024] = True
    hit[2304:2560] = True
    assert m[hit].isnan().all() and v[hit].isnan().all()
    for x, y in zip((m, v), ob.onebit_adamw8_get_state(*b.state)):
        assert torch.equal(x[~hit], y[~hit])
    assert a.p[0][[777, 2499]].isnan().all()
    a.p[0][[777, 2499]] = b.p[0][[777, 2499]]
    assert same_bits([a.p_arena], [b.p_arena])


@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
@pytest.mark.parametrize("size", [1e18, 1e4, 60.0, 1e-12, 1e-18, 0.0])
def test_sizes_of_gradients(size, eight):
    """Gradients from where their squares are near fp32's largest value to where they are below its
    smallest: the moments keep the accuracy of their operations."""
    pr = Problem([5000, 100], torch.float32, torch.float32, 1, seed=8, eight=eight)
    for i, g in enumerate(pr.g):
        g.copy_(torch.randn(g.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(i))
                * size)
    for x in pr.state:
        x.zero_()
    pr.inside[:] = True                            # the places behind were just zeroed
    check_step(pr, None, 1)
    check_step(pr, None, 2)


@pytest.mark.parametrize("align", [1, 16])
def test_8_bit_states_at_every_power_of_two(align):
    """One tensor of whole and one of odd length for each size of gradients from 2^-70 to 2^50, so
    that the blocks' exponents pass every border of the kernel's fast form, from fresh states on;
    some blocks hold a single value."""
    powers = list(range(-70, 51))
    sizes = [n for _ in powers for n in (1024, 300)]
    pr = Problem(sizes, torch.float32, torch.float32, align, seed=21, eight=True)
    gen = torch.Generator(DEV).manual_seed(5)
    for x in pr.state:
        x.zero_()
    pr.inside[:] = True
    for t in (1, 2, 3):
        for i, g in enumerate(pr.g):
            g.copy_(torch.randn(g.shape, device=DEV, generator=gen) * 2.0 ** powers[i // 2])
            g[256:511] = 0.0
        check_step(pr, None, t)


def test_v_above_zero_never_reads_as_zero():
    """A block with one large and many tiny gradients: v of the tiny ones stays above 0, so that no
    later denominator is eps alone, and exact zeros stay 0."""
    n = 4096
    p = torch.zeros(n, device=DEV)
    g = torch.full((n,), 1e-9, device=DEV)
    g[::256] = 1.0
    g[7::256] = 0.0
    opt = ob.AdamW([p], weight_decay=0.0, state="q8")
    for _ in range(4):
        opt.step([p], [g], 1e-3)
    m, v = opt.get_state()
    assert (v[7::256] == 0).all() and (m[7::256] == 0).all()
    rest = g == g[1]
    assert (v[rest] > 0).all()
    assert p[rest].abs().max() <= 4 * 1e-3 * 1.001


def test_more_than_2_to_31_elements_32():
    n = (1 << 31) + 300
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB of free device memory")
    p, g = (torch.zeros(n, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    total = ob.onebit_adamw_layout([n])[1]
    m, v = (torch.zeros(total, device=DEV) for _ in range(2))
    ctl = torch.zeros(8, dtype=torch.int64, device=DEV)
    tail = 70_000
    g[-tail:] = (torch.randn(tail, device=DEV) * 1e-2).to(torch.bfloat16)
    ob.onebit_adamw_step([p], [g], m, v, ctl, 1e-2)
    (p1, m1, v1), (ep, em, ev) = ref.step64(host(p[-tail:]) * 0, host(g[-tail:]), np.zeros(tail),
                                            np.zeros(tail), 1, 1e-2, 0.9, 0.999, 1e-8, 0.0)
    assert (np.abs(host(m[n - tail:n]) - m1) <= em).all()
    assert (np.abs(host(v[n - tail:n]) - v1) <= ev).all()
    assert (np.abs(host(p[-tail:]) - p1) <= ref.bf16_bound(p1, ep)).all()
    assert not p[:-tail].any() and not m[:n - tail].any() and not m[n:].any()


def test_more_than_2_to_31_elements():
    n = (1 << 31) + 300
    if torch.cuda.mem_get_info()[0] < 20e9:
        pytest.skip("needs 20 GB of free device memory")
    p = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    tail = 70_000
    g[-tail:] = (torch.randn(tail, device=DEV) * 1e-2).to(torch.bfloat16)
    g[:tail] = g[-tail:]
    offsets, total = ob.onebit_adamw_layout([n])
    state = [torch.zeros(k, dtype=torch.uint8, device=DEV)
             for k in (total, total, total // BLOCK, total // BLOCK)]
    ctl = torch.zeros(8, dtype=torch.int64, device=DEV)
    ob.onebit_adamw8_step([p], [g], *state, ctl, 1e-2, seed=3)
    norm, _ = ob.onebit_grad_norm([g])
    want = math.sqrt(2 * float(g[-tail:].double().square().sum()))
    assert abs(float(norm) - want) <= want * 2 ** -23
    assert not p[tail:-tail].any()
    # the first step moves every element with a gradient by lr, to bf16's rounding and eps
    moved = p[-tail:][g[-tail:].abs() > 1e-4].abs().float()
    assert ((moved - 1e-2).abs() <= 1e-2 * (2 ** -8 + 2e-4)).all()
    start = n - tail - (n - tail) % BLOCK
    words = ref.random_words(np.arange(start, total), 3, 1)
    gt = np.zeros(total - start)
    gt[:n - start] = host(g[start:])
    m32, v32 = ref.moments32(gt, gt * 0, gt * 0, 0.9, 0.999)
    for x, codes, exps, signed, r in ((m32, state[0], state[2], True, words >> 16),
                                      (v32, state[1], state[3], False, words & 0xFFFF)):
        want_c, want_k = ref.encode64(x, signed, r / 65536)
        assert np.array_equal(codes[start:].cpu().numpy()[:n - start], want_c[:n - start])
        assert np.array_equal(exps[start // BLOCK:].cpu().numpy(), want_k)


# ----------------------------------------------------------------------------------------------
# the 8-bit states' values

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_code_at_every_exponent(dtype):
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(256)
    exps = torch.arange(256, dtype=torch.uint8, device=DEV)
    m, v = ob.onebit_adamw8_get_state(codes, codes, exps, exps, dtype=dtype)
    for got, signed in ((m, True), (v, False)):
        want = ref.decode64(codes.cpu().numpy(), exps.cpu().numpy(), signed)
        with np.errstate(over="ignore"):
            want = torch.from_numpy(want.astype(np.float32)).to(dtype)
        assert torch.equal(got.cpu().nan_to_num(-5.0), want.nan_to_num(-5.0))
        assert torch.equal(got.cpu().isnan(), want.isnan())


def test_set_state_rounds_to_nearest_even_and_gives_back_what_get_gave():
    rng = np.random.default_rng(0)
    blocks = 300
    scale = np.repeat(np.ldexp(1.0, rng.integers(-150, 126, blocks)), BLOCK)
    x = (rng.standard_normal(blocks * BLOCK) * scale * np.exp2(-rng.random(blocks * BLOCK) * 30))
    x = np.clip(x, -3.1e38, 3.1e38).astype(np.float32)
    x[5 * BLOCK:6 * BLOCK] = 0.0
    x[6 * BLOCK:7 * BLOCK:3] = np.float32(1e-45)
    # halfway between two codes, below the largest code and just above it
    x[7 * BLOCK:8 * BLOCK] = 0.0
    x[7 * BLOCK:7 * BLOCK + 6] = [1.875, 1.0625, 1.1875, -1.0625, 1.4375, 2.0 ** -20]
    x[8 * BLOCK:9 * BLOCK] = 0.0
    x[8 * BLOCK] = np.nextafter(np.float32(1.875), np.float32(2))
    x[9 * BLOCK] = np.inf
    x[10 * BLOCK + 9] = np.nan
    x[11 * BLOCK + 255] = 3.3e38                       # above 1.875 * 2^127
    xs = torch.from_numpy(x).to(DEV)
    va = torch.from_numpy(np.where(np.isnan(x), x, np.maximum(x, 0))).to(DEV)
    codes = [torch.zeros(blocks * BLOCK, dtype=torch.uint8, device=DEV) for _ in range(2)]
    exps = [torch.zeros(blocks, dtype=torch.uint8, device=DEV) for _ in range(2)]
    ob.onebit_adamw8_set_state(*codes, *exps, xs, xs)   # v: below 0 counts as 0
    for i, (y, signed) in enumerate(((xs, True), (va, False))):
        want_c, want_k = ref.encode64(host(y), signed)
        assert np.array_equal(exps[i].cpu().numpy(), want_k)
        assert np.array_equal(codes[i].cpu().numpy(), want_c)
    assert exps[0][9:12].tolist() == [255] * 3
    m, v = ob.onebit_adamw8_get_state(*codes, *exps)
    fine = ~m.isnan()
    # rounded to nearest: half a step, which is 1/16 of the value's binade or the smallest step's
    # (there the value was rounded once before, to 2^-20 of a step)
    half = np.ldexp(1 + 2 ** -19, exps[0].cpu().numpy().astype(int) - 127 - 18)
    least = torch.from_numpy(np.repeat(half, BLOCK)).to(DEV)
    err = (m.double() - xs.double()).abs()[fine]
    assert (err <= torch.maximum(xs.double().abs() / 16, least)[fine]).all()
    again = [torch.zeros_like(t) for t in codes + exps]
    ob.onebit_adamw8_set_state(*again, m, v)
    m2, v2 = ob.onebit_adamw8_get_state(*again)
    assert same_bits([m2[fine], v2[~v.isnan()]], [m[fine], v[~v.isnan()]])
    assert m2[~fine].isnan().all()


def test_stochastic_rounding_keeps_the_mean():
    """beta2 = 0.999 moves v by a thousandth of itself a step, a sixtieth of the codes' spacing:
    the mean of v over many elements follows the exact recurrence all the same. Stationary standard
    deviation of one element: at most 25 % (half the largest spacing, 1/8, under the root); the mean
    over n independent elements is within 5 / sqrt(n) of that, plus the 16 bits' bias: 2^-17 of a
    spacing every step, at most 2^-17 / 8 / (1 - beta2) = 0.1 % in all. The largest element of each
    block is left out: it defines the exponent."""
    n, steps = 1 << 18, 400
    p = torch.zeros(n, device=DEV)
    opt = ob.AdamW([p], weight_decay=0.0, state="q8", seed=11)
    g = torch.full((n,), 0.5, device=DEV)
    g[::256] = 2.0
    m0 = torch.zeros(n, device=DEV)
    v0 = torch.full((n,), 1.0, device=DEV)
    v0[::256] = 8.0
    opt.set_state(m0, v0, 1000)
    for _ in range(steps):
        opt.step([p], [g], 0.0)
    m, v = opt.get_state()
    rest = g == 0.5
    k = int(rest.sum())
    want_v = 0.999 ** steps * 1.0 + (1 - 0.999 ** steps) * 0.25
    assert abs(float(v[rest].double().mean()) / want_v - 1) <= 5 * 0.25 / math.sqrt(k) + 1e-3
    # m: noise of at most half a spacing (1/16) a step, sqrt(1 / (1 - 0.81)) of it in all
    want_m = (1 - 0.9 ** steps) * 0.5
    bound = 5 * 2.3 / 16 / math.sqrt(k) + 2 ** -17 / 8 / 0.1
    assert abs(float(m[rest].double().mean()) / want_m - 1) <= bound
    assert float(v[rest].std()) > 0                  # elements differ: the bits are their own


# ----------------------------------------------------------------------------------------------
# the gradient norm

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,align", [(SHORT, 16), (SHORT, 1), (LONG, 8), (LONGER, 1), ([1], 1),
                                         ([2_000_003], 16)],
                         ids=["short", "short_odd", "130", "1700", "one", "2M"])
def test_grad_norm(sizes, align, dtype):
    pr = Problem(sizes, torch.float32, dtype, align, seed=9)
    want = math.sqrt(sum(float((host(g) ** 2).sum()) for g in pr.g))
    work = torch.zeros(16384, dtype=torch.uint8, device=DEV)
    for max_norm in (want * 0.25, want * 4, math.inf):
        norm, scale = ob.onebit_grad_norm(pr.g, max_norm, work)
        # fp64 sums: nothing next to the result's own rounding
        assert abs(float(norm) - want) <= want * 2 ** -24 * 1.01
        s = min(1.0, max_norm / want)
        assert abs(float(scale) - s) <= s * 2 ** -24 * 1.01
    first = [x.clone() for x in ob.onebit_grad_norm(pr.g, 1.0, work)]
    for _ in range(3):
        assert same_bits(first, ob.onebit_grad_norm(pr.g, 1.0))


def test_grad_norm_over_lists_of_different_types():
    a = Problem(SHORT, torch.float32, torch.float32, 1, seed=1)
    b = Problem(LONGER, torch.float32, torch.bfloat16, 8, seed=2)
    work = torch.zeros(16384, dtype=torch.uint8, device=DEV)
    ob.onebit_grad_norm(a.g, 1.0, work)
    norm, scale = ob.onebit_grad_norm(b.g, 1.0, work, accumulate=True)
    sumsq = sum(float((host(g) ** 2).sum()) for g in a.g + b.g)
    assert abs(float(norm) - math.sqrt(sumsq)) <= math.sqrt(sumsq) * 2 ** -24 * 1.01
    assert abs(float(work[:8].view(torch.float64)) - sumsq) <= sumsq * 1e-12
    # and nothing added: the same norm, another limit
    norm, scale = ob.onebit_grad_norm([], 0.5 * math.sqrt(sumsq), work, accumulate=True)
    assert abs(float(scale) - 0.5) <= 2 ** -24
    norm, scale = ob.onebit_grad_norm([], 1.0, work)
    assert float(norm) == 0.0 and float(scale) == 1.0


@pytest.mark.parametrize("value,norm,scale", [
    (1e30, 1e30 * math.sqrt(1000), 1 / (1e30 * math.sqrt(1000))), (1e-30, 1e-30 * math.sqrt(1000), 1.0),
    (0.0, 0.0, 1.0), (math.inf, math.inf, math.nan), (math.nan, math.nan, math.nan),
    (3e38, math.inf, math.nan)])
def test_grad_norm_extremes(value, norm, scale):
    """Squares beyond fp32's range on either side do not matter; a norm that is not a finite fp32
    number gives a scale of NaN, which leaves the step out."""
    got_norm, got_scale = ob.onebit_grad_norm([torch.full((1000,), value, device=DEV)], 1.0)
    for got, want in ((float(got_norm), norm), (float(got_scale), scale)):
        if math.isfinite(want):
            # the fp32 input and result: two roundings
            assert abs(got - want) <= abs(want) * 2 ** -23 + 2.0 ** -149
        else:
            assert got == want or (math.isnan(got) and math.isnan(want))


# ----------------------------------------------------------------------------------------------
# refusals that need device tensors

def test_refusals_on_the_device():
    pr = Problem([1000, 300], torch.float32, torch.float32)
    m, v = pr.state
    before = pr.everything()
    flat = torch.zeros(8, 8, device=DEV)

    def step(p=pr.p, g=pr.g, m=m, v=v, ctl=pr.ctl, lr=1e-3, **kw):
        return lambda: ob.onebit_adamw_step(p, g, m, v, ctl, lr, **kw)
    for call, kind, why in [
            (step(p=[flat.t()], g=[flat]), ValueError, "contiguous"),
            (step(g=[x.half() for x in pr.g]), TypeError, "float32 or bfloat16"),
            (step(g=[pr.g[0], pr.g[1].bfloat16()]), ValueError, "one type"),
            (step(g=[pr.g[0], pr.g[1].cpu()]), ValueError, "one device"),
            (step(g=pr.g[::-1]), ValueError, "lengths"),
            (step(g=pr.g[:1]), ValueError, "gradients"),
            (step(m=m[:-1]), ValueError, "m holds"),
            (step(v=v.double()), TypeError, "v must be"),
            (step(ctl=pr.ctl[:4]), ValueError, "ctl holds"),
            (step(lr=torch.zeros(1, device=DEV)), TypeError, "lr must be"),
            (step(grad_scale=torch.zeros(1, dtype=torch.float64, device=DEV)), TypeError, "scale"),
            (step(copies=[x.clone() for x in pr.p]), TypeError, "copies must be"),
            (step(weight_decay=[0.1]), ValueError, "weight decays"),
            (step(p=[pr.p[0], pr.p[0][:300]]), ob.OneBitError, "overlap"),
            (step(g=[pr.p[0], pr.g[1]]), ob.OneBitError, "overlap"),
            (step(m=v), ob.OneBitError, "overlap"),
            (step(weight_decay=-1.0), ob.OneBitError, "decay")]:
        with pytest.raises(kind, match=why):
            call()
    opt = ob.AdamW(pr.p, max_norm=1.0)
    with pytest.raises(ValueError, match="exclude"):
        opt.step(pr.p, pr.g, 1e-3, grad_scale=torch.ones(1, device=DEV))
    with pytest.raises(ValueError, match="optimizer's"):
        opt.step(pr.p[::-1], pr.g[::-1], 1e-3)
    with pytest.raises(ob.OneBitError, match="max_norm"):
        ob.AdamW(pr.p, max_norm=-1.0).step(pr.p, pr.g, 1e-3)
    with pytest.raises(ValueError, match="multiple of 256"):
        ob.onebit_adamw8_get_state(*[torch.zeros(100, dtype=torch.uint8, device=DEV)] * 4)
    torch.cuda.synchronize()
    assert same_bits(before, pr.everything())
    # gradients may share memory
    pr.step(grads=[pr.g[0], pr.g[0][:300]])


def test_autograd_sees_that_parameters_changed():
    """The step counts as an in-place change of the parameters: a backward pass through values that
    it overwrote is refused by autograd."""
    w = torch.randn(1000, device=DEV, requires_grad=True)
    loss = (w * w).sum()
    opt = ob.AdamW([w])
    g = torch.ones_like(w)
    with torch.no_grad():
        opt.step([w], [g], 1e-3)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


# ----------------------------------------------------------------------------------------------
# streams, graphs, and the operators together

@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
def test_another_stream(eight):
    """Work queued on a stream that is not the current one, the gradients dropped at once and their
    memory handed out again and overwritten."""
    a = Problem([1 << 20], torch.float32, torch.float32, seed=1, eight=eight)
    b = Problem([1 << 20], torch.float32, torch.float32, seed=1, eight=eight)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(1000)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)               # some milliseconds: the step begins later
    grads = [a.g[0].clone()]
    side.wait_stream(torch.cuda.current_stream())
    a.step(stream=side, grads=grads)
    del grads
    junk = [torch.full((1 << 20,), math.nan, device=DEV) for _ in range(4)]
    side.synchronize()
    b.step()
    assert same_bits(a.everything(), b.everything())
    a.step(stream=side.cuda_stream)
    b.step()
    torch.cuda.synchronize()
    assert same_bits(a.everything(), b.everything()) and junk


@pytest.mark.parametrize("state", ["f32", "q8"])
def test_a_captured_step_replayed(state):
    """Norm, clip and step in one graph: every replay is the next step, with the learning rate that
    its tensor holds then; a replay whose norm is not finite is left out."""
    sizes = [700, 5, 0, 66_000]
    gen = torch.Generator(device=DEV).manual_seed(3)
    start = [torch.randn(n, device=DEV, generator=gen) for n in sizes]
    draws = [[torch.randn(n, device=DEV, generator=gen) for n in sizes] for _ in range(4)]
    draws[2][3][1234] = math.nan
    lrs = [1e-3, 5e-4, 2e-4, 1e-4]

    def fresh():
        p = [x.clone() for x in start]
        return p, [x.to(torch.bfloat16) for x in p], ob.AdamW(p, max_norm=1.0, state=state, seed=4)
    pe, ce, eager = fresh()
    for g, lr in zip(draws, lrs):
        eager.step(pe, g, lr, copies=ce)
    pg, cg, opt = fresh()
    g = [torch.zeros(n, device=DEV) for n in sizes]
    lr = torch.zeros(1, dtype=torch.float64, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        opt.step(pg, g, lr, copies=cg)
    assert opt.counts() == (0, 0)                    # capturing runs nothing
    for new, rate in zip(draws, lrs):
        for x, y in zip(g, new):
            x.copy_(y)
        lr.fill_(rate)
        graph.replay()
    torch.cuda.synchronize()
    assert opt.counts() == (3, 1) == eager.counts()
    assert same_bits(pe + ce + list(eager.get_state()) + [eager.ctl[:4]],
                     pg + cg + list(opt.get_state()) + [opt.ctl[:4]])
    del graph


@pytest.mark.parametrize("state", ["f32", "q8"])
def test_a_run_with_clipping_a_checkpoint_and_a_change_of_state_width(state):
    """A small least-squares model trained as a user would: norm, clip, step, checkpoint, resume
    (bit for bit), go on with states of the other width. The parameters follow the 64-bit AdamW
    exactly as far as the bound of each step allows, with the states of each step taken over."""
    gen = torch.Generator(device=DEV).manual_seed(6)
    w = [(torch.randn(40, 30, device=DEV, generator=gen) * 0.1).requires_grad_(),
         torch.zeros(30, device=DEV).requires_grad_()]
    x = torch.randn(256, 40, device=DEV, generator=gen)
    y = torch.randn(256, 30, device=DEV, generator=gen)
    opt = ob.AdamW(w, weight_decay=[0.1, 0.0], max_norm=0.5, state=state, seed=2)

    def grads(params):
        return torch.autograd.grad(((x @ params[0] + params[1] - y) ** 2).sum(), params)

    def run(o, params, count):
        for _ in range(count):
            o.step([t.detach() for t in params], grads(params), 1e-3)
    for k in range(3):
        g = grads(w)
        p0, g0 = [host(t).ravel() for t in w], [host(t).ravel() for t in g]
        m0, v0 = (host(t) for t in opt.get_state())
        norm = math.sqrt(sum((t ** 2).sum() for t in g0))
        opt.step([t.detach() for t in w], g, 1e-3)
        assert abs(float(opt.norm) - norm) <= norm * 2 ** -24 * 1.01
        scale = float(np.float32(min(1.0, 0.5 / norm)))
        for i, (o, n) in enumerate(zip(opt.offsets, opt.lengths)):
            (p1, _, _), (ep, _, _) = ref.step64(p0[i], g0[i], m0[o:o + n], v0[o:o + n], k + 1, 1e-3,
                                                0.9, 0.999, 1e-8, [0.1, 0.0][i], scale)
            # the kernel's scale may be the fp32 next to this one: both moments move by that much
            (pa, _, _), _ = ref.step64(p0[i], g0[i], m0[o:o + n], v0[o:o + n], k + 1, 1e-3, 0.9,
                                       0.999, 1e-8, [0.1, 0.0][i], scale * (1 + 2 ** -23))
            assert (np.abs(host(w[i]).ravel() - p1) <= ep + np.abs(pa - p1)).all()
    ck, saved = opt.checkpoint(), [t.detach().clone() for t in w]
    run(opt, w, 3)
    other = ob.AdamW(saved, weight_decay=[0.1, 0.0], max_norm=0.5, state=state, seed=2)
    other.restore(ck)
    again = [t.requires_grad_() for t in saved]
    run(other, again, 3)
    assert same_bits([t.detach() for t in w], [t.detach() for t in again])
    assert other.counts() == (6, 0)
    # the other width: 8 bits into 32 exactly, 32 into 8 to half a step
    swapped = ob.AdamW(again, weight_decay=[0.1, 0.0], max_norm=0.5,
                       state="q8" if state == "f32" else "f32", seed=2)
    m, v = other.get_state()
    swapped.set_state(m, v, 6)
    m2, v2 = swapped.get_state()
    if state == "q8":
        assert same_bits([m2, v2], [m, v])
    else:
        k = m.view(-1, BLOCK).abs().amax(1, keepdim=True) * 2.0 ** -17
        assert ((m2 - m).abs().view(-1, BLOCK) <= torch.maximum(m.abs().view(-1, BLOCK) / 16, k)).all()
    run(swapped, again, 2)
    assert swapped.counts() == (8, 0)
    assert all(torch.isfinite(t).all() for t in again)
    with pytest.raises(ValueError, match="another kind"):
        swapped.restore(ck)
