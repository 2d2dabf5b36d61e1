"""``AdamW``'s states on their way in and out: what lies behind a tensor, refusals that change
nothing, and checkpoints."""
import math

import numpy as np
import pytest
import torch

import communication_compressed_optimizer_momentum_b200 as ob
import adamw_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BLOCK = 256
SIZES = [1, 255, 256, 0, 257, 700, 512]


def params(sizes=SIZES):
    return [torch.zeros(n, device=DEV) for n in sizes]


def moments(opt, seed=0):
    """Flat moments with zeros behind the tensors, and where the tensors' own places are."""
    rng = np.random.default_rng(seed)
    inside = np.zeros(opt.total, bool)
    for o, n in zip(opt.offsets, opt.lengths):
        inside[o:o + n] = True
    m = np.where(inside, rng.standard_normal(opt.total) * 1e-2, 0.0).astype(np.float32)
    v = np.where(inside, rng.random(opt.total) * 1e-4, 0.0).astype(np.float32)
    return m, v, inside


@pytest.mark.parametrize("junk", [math.nan, math.inf, 1e30, 77.0])
@pytest.mark.parametrize("state", ["q8", "f32"])
def test_what_lies_behind_a_tensor_does_not_count(state, junk):
    """Moments whose places behind the tensors hold anything: the tensors' elements become what they
    become with zeros there, the caller's vectors stay as they are, and the next step is the same."""
    opt, other = (ob.AdamW(params(), state=state, seed=1) for _ in range(2))
    m, v, inside = moments(opt)
    dirty = [torch.from_numpy(np.where(inside, x, np.float32(junk))).to(DEV) for x in (m, v)]
    kept = [x.clone() for x in dirty]
    opt.set_state(*dirty, 3)
    assert all(torch.equal(x.view(torch.int32), y.view(torch.int32)) for x, y in zip(dirty, kept))
    clean = [torch.from_numpy(x).to(DEV) for x in (m, v)]
    other.set_state(*clean, 3)
    for x, y, want, signed in zip(opt.get_state(), other.get_state(), (m, v), (True, False)):
        x, y = x.cpu().numpy(), y.cpu().numpy()
        assert np.array_equal(x[inside], y[inside])
        if state == "q8":
            codes, k = ref.encode64(want, signed)
            assert np.array_equal(x[inside], ref.decode64(codes, k, signed)[inside])
    gen = torch.Generator(device=DEV).manual_seed(2)
    grads = [torch.randn(n, device=DEV, generator=gen) for n in SIZES]
    p, q = params(), params()
    opt.step(p, grads, 1e-2)
    other.step(q, grads, 1e-2)
    assert all(torch.equal(x, y) for x, y in zip(p, q))
    assert all(torch.isfinite(x).all() for x in p)


@pytest.mark.parametrize("sizes", [SIZES, [512, 256]], ids=["gaps", "whole_blocks"])
@pytest.mark.parametrize("state", ["q8", "f32"])
def test_moments_at_any_address(state, sizes):
    """Views at addresses that are aligned to one element only, as in a loaded checkpoint."""
    opt, other = (ob.AdamW(params(sizes), state=state) for _ in range(2))
    m, v, _ = moments(opt, 4)
    arena = torch.full((2 * opt.total + 4,), 5.0, device=DEV)
    views = [arena[1:1 + opt.total], arena[opt.total + 3:2 * opt.total + 3]]
    clean = [torch.from_numpy(x).to(DEV) for x in (m, v)]
    for x, y in zip(views, clean):
        assert x.data_ptr() % 16 != 0
        x.copy_(y)
    opt.set_state(*views, 9)
    other.set_state(*clean, 9)
    assert all(torch.equal(x, y) for x, y in zip(opt.get_state(), other.get_state()))
    assert opt.counts() == other.counts() == (9, 0)


@pytest.mark.parametrize("state", ["q8", "f32"])
def test_moments_of_any_shape(state):
    """Contiguous moments count as flat whatever their shape, and longer ones from their start."""
    sizes = [300, 256]
    opt, other = (ob.AdamW(params(sizes), state=state) for _ in range(2))
    m, v, _ = moments(opt, 5)
    clean = [torch.from_numpy(x).to(DEV) for x in (m, v)]
    other.set_state(*clean, 2)
    opt.set_state(clean[0].view(-1, 256), torch.cat([clean[1], clean[1]]).view(2, -1), 2)
    assert all(torch.equal(x, y) for x, y in zip(opt.get_state(), other.get_state()))
    opt.set_state(torch.cat([clean[0], clean[0]]).view(-1, 2), clean[1].view(-1, 1), 2)
    assert all(torch.equal(x, y) for x, y in zip(opt.get_state(), other.get_state()))


def test_a_refused_set_state_changes_nothing():
    """Moments that lie in the states themselves, which the encoder refuses: the step count stays."""
    opt = ob.AdamW(params([512, 2048]), state="q8")
    m, v, _ = moments(opt)
    opt.set_state(torch.from_numpy(m).to(DEV), torch.from_numpy(v).to(DEV), 6)
    # 2560 codes and, as fp32, the same memory: a buffer that both begin in
    arena = torch.zeros(4 * opt.total, dtype=torch.uint8, device=DEV)
    arena[:opt.total] = opt.m
    opt.m = arena[:opt.total]
    before = [x.clone() for x in (*opt._state(), opt.ctl)]
    with pytest.raises(ob.OneBitError, match="overlap"):
        opt.set_state(arena.view(torch.float32), torch.from_numpy(v).to(DEV), 11)
    assert opt.counts() == (6, 0)
    assert all(torch.equal(x, y) for x, y in zip(before, (*opt._state(), opt.ctl)))
    with pytest.raises(ValueError, match="holds"):
        opt.set_state(torch.from_numpy(m).to(DEV)[:-1], torch.from_numpy(v).to(DEV), 11)
    assert opt.counts() == (6, 0)


@pytest.mark.parametrize("side", [False, True], ids=["current", "side"])
@pytest.mark.parametrize("state", ["q8", "f32"])
def test_a_refused_clipped_step_changes_nothing(state, side):
    """Whatever the step refuses, it refuses before the norm of its gradients is taken."""
    n = 5000
    arena = torch.zeros(2 * n + 4096, device=DEV)
    p = [arena[:n], arena[n:2 * n]]
    g = [torch.randn(n, device=DEV) for _ in p]
    opt = ob.AdamW(p, weight_decay=0.01, max_norm=1.0, state=state)
    opt.step(p, g, 1e-2)
    norm = float(opt.norm)
    assert abs(norm - float(torch.cat(g).double().norm())) <= 1e-6 * norm
    torch.cuda.synchronize()
    before = [x.clone() for x in (arena, opt.work, opt.ctl, *opt._state())]
    versions = [x._version for x in p]
    other = [x * 2 for x in g]
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()

    def refused(why, params=p, lr=1e-2, **change):
        kept = {name: getattr(opt, name) for name in change}
        for name, x in change.items():
            setattr(opt, name, x)
        with pytest.raises(ob.OneBitError, match=why):
            opt.step(params, other, lr, stream=stream)
        for name, x in kept.items():
            setattr(opt, name, x)
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(-1).view(torch.uint8), y.view(-1).view(torch.uint8))
                   for x, y in zip(before, (arena, opt.work, opt.ctl, *opt._state())))
        assert float(opt.norm) == norm and [x._version for x in p] == versions
    refused("lr", lr=math.nan)
    refused("beta", beta2=1.0)
    refused("eps", eps=-1.0)
    refused("decay", weight_decay=-0.1)
    refused("max_norm", max_norm=-1.0)
    refused("overlap", params=[p[0], p[0]])
    refused("overlap", params=[p[0], other[1]])
    refused("overlap", ctl=arena[:16].view(torch.int64))
    # a norm's buffer that begins among the parameters' last elements and ends behind them
    refused("overlap", work=arena[2 * n - 64:2 * n + 4032].view(torch.uint8))
    opt.step(p, other, 1e-2)
    assert float(opt.norm) == pytest.approx(2 * norm, rel=1e-6) and opt.counts() == (2, 0)


@pytest.mark.parametrize("seed", [5, -1, (1 << 63) + 12345, (1 << 64) + 7])
def test_a_checkpoint_continues_bit_for_bit_whatever_the_other_seed(seed, tmp_path):
    """8-bit states: the rounding's seed is part of a checkpoint, saved and loaded like the rest; one
    without it (or of 32-bit states, which round nothing at random) leaves the optimizer's own."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    grads = [[torch.randn(n, device=DEV, generator=gen) for n in SIZES] for _ in range(4)]
    p = params()
    opt = ob.AdamW(p, state="q8", seed=seed)
    opt.step(p, grads[0], 1e-2)
    opt.step(p, grads[1], 1e-2)
    torch.save(opt.checkpoint(), tmp_path / "ck.pt")
    q = [x.clone() for x in p]
    other = ob.AdamW(q, state="q8", seed=99)
    other.restore(torch.load(tmp_path / "ck.pt"))
    for g in grads[2:]:
        opt.step(p, g, 1e-2)
        other.step(q, g, 1e-2)
    for x, y in zip((*p, *opt._state(), opt.ctl), (*q, *other._state(), other.ctl)):
        assert torch.equal(x, y)
    ck = opt.checkpoint()
    assert {k: v.cpu() for k, v in ck.items()}.keys() == ck.keys()
    del ck["seed"]
    third = ob.AdamW(q, state="q8", seed=42)
    third.restore(ck)
    assert third.seed == 42 and third.counts() == (4, 0)
    narrow = ob.AdamW(q, state="f32", seed=42)
    assert "seed" not in narrow.checkpoint()
    with pytest.raises(ValueError, match="another kind"):
        narrow.restore(opt.checkpoint())


@pytest.mark.parametrize("state", ["q8", "f32"])
def test_moments_that_require_gradients_leave_states_that_do_not(state):
    """A set_state is not part of anyone's graph."""
    opt = ob.AdamW(params(), state=state)
    m, v, _ = moments(opt, 7)
    given = [torch.from_numpy(x).to(DEV).requires_grad_() for x in (m, v)]
    opt.set_state(*given, 4)
    assert not any(x.requires_grad for x in (*opt._state(), opt.ctl, *opt.get_state()))
    ck = opt.checkpoint()
    ck["m"] = ck["m"].float().requires_grad_().to(ck["m"].dtype)
    other = ob.AdamW(params(), state=state)
    other.restore(ck)
    assert not any(x.requires_grad for x in (*other._state(), *other.checkpoint().values()))
