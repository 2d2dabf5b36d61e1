"""The AdamW functions and ``AdamW`` on a stream that is not the current one: results are that
stream's memory, never a block that work queued on the current stream still uses."""
import math

import pytest
import torch

import communication_compressed_optimizer_momentum_b200 as ob

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BLOCK = 256
PAUSE = 20_000_000                       # cycles: some milliseconds of a busy stream


def states(n, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    codes = [torch.randint(0, 256, (n,), dtype=torch.uint8, device=DEV, generator=gen)
             for _ in range(2)]
    exps = [torch.full((n // BLOCK,), k, dtype=torch.uint8, device=DEV) for k in (118, 110)]
    return codes + exps


def delayed_copies(n, dtype, count=4):
    """Values, copies of them that the current stream takes some milliseconds from now, and no
    other reference to what the copies are made from: its memory is free for that stream again."""
    values = [torch.randn(n, device=DEV).to(dtype) for _ in range(count)]
    kept = [x.cpu() for x in values]
    torch.cuda._sleep(PAUSE)
    copies = [x.clone() for x in values]
    return kept, copies


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_get_state_takes_the_memory_of_its_stream(dtype):
    n = 1 << 20
    state = states(n)
    want = ob.onebit_adamw8_get_state(*state, dtype=dtype)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept, copies = delayed_copies(n, dtype)
    got = ob.onebit_adamw8_get_state(*state, dtype=dtype, stream=side)
    side.synchronize()
    assert all(torch.equal(x.cpu(), y.cpu()) for x, y in zip(got, want))
    assert all(torch.equal(x.cpu(), y) for x, y in zip(copies, kept))


@pytest.mark.parametrize("by", ["stream", "handle"])
def test_results_may_be_dropped_while_the_current_stream_reads_them(by):
    """A result is the other stream's memory, which that stream would hand out again at once if it
    were not marked as used on the current one."""
    n = 1 << 20
    state = states(n, 1)
    grads = [torch.randn(5000, device=DEV)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    stream = side if by == "stream" else side.cuda_stream
    m, v = ob.onebit_adamw8_get_state(*state, stream=stream)
    norm, scale = ob.onebit_grad_norm(grads, 1.0, stream=stream)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(PAUSE)
    copies = [x.clone() for x in (m, v, norm, scale)]
    del m, v, norm, scale
    with torch.cuda.stream(side):
        junk = [torch.full((n,), math.nan, device=DEV) for _ in range(4)]
        junk += [torch.full((16384,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
    want = list(ob.onebit_adamw8_get_state(*state)) + list(ob.onebit_grad_norm(grads, 1.0))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(copies, want)) and junk


def busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(PAUSE)


@pytest.mark.parametrize("by", ["stream", "handle"])
@pytest.mark.parametrize("state", ["q8", "f32"])
def test_everything_of_an_optimizer_on_one_other_stream(state, by):
    """A clipped step, a checkpoint, another step, its moments, the checkpoint restored and the moments
    set, all queued on a stream that is busy for some milliseconds, with no wait between the calls and
    the inputs dropped at once: what they give is what the same calls on the current stream give."""
    sizes = [70_001, 300, 0, 1 << 18]
    gen = torch.Generator(device=DEV).manual_seed(3)
    start = [torch.randn(n, device=DEV, generator=gen) for n in sizes]
    draws = [[torch.randn(n, device=DEV, generator=gen) for n in sizes] for _ in range(3)]

    def run(side):
        stream = side if by == "stream" or side is None else side.cuda_stream
        p = [x.clone() for x in start]
        opt = ob.AdamW(p, weight_decay=0.01, max_norm=1.0, state=state, seed=9)
        given = torch.rand(2, opt.total, device=DEV, generator=torch.Generator(DEV).manual_seed(8))
        grads = [[x.clone() for x in g] for g in draws]
        out = []
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
            busy(side)
        opt.step(p, grads.pop(0), 1e-2, stream=stream)
        ck = opt.checkpoint(stream=stream)
        opt.step(p, grads.pop(0), 1e-2, stream=stream)
        m, v = opt.get_state(stream=stream)
        if side is not None:
            with torch.cuda.stream(side):                 # 32-bit states: they are the states
                out += [m.clone(), v.clone()]
        else:
            out += [m.clone(), v.clone()]
        opt.restore(ck, stream=stream)
        opt.step(p, grads.pop(0), 1e-2, stream=stream)
        after = opt.checkpoint(stream=stream)
        opt.set_state(given[0], given[1], 40, stream=stream)
        del given, m, v
        if side is not None:
            junk = [torch.full((opt.total,), math.nan, device=DEV) for _ in range(4)]
            assert junk
        assert opt.counts() == (40, 0)
        out += [ck[n] for n in sorted(ck)] + [after[n] for n in sorted(after)] + p
        out += [*opt._state(), opt.ctl, opt.norm]
        torch.cuda.synchronize()
        return out
    want, got = run(None), run(torch.cuda.Stream())
    assert len(want) == len(got)
    for i, (x, y) in enumerate(zip(got, want)):
        assert torch.equal(x.reshape(-1).view(torch.uint8), y.reshape(-1).view(torch.uint8)), i


def test_counts_waits_for_the_device():
    p, g = [torch.zeros(1000, device=DEV)], [torch.ones(1000, device=DEV)]
    opt = ob.AdamW(p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy(side)
    opt.step(p, g, 1e-3, stream=side)
    assert opt.counts() == (1, 0)


def test_a_checkpoint_is_the_memory_of_its_stream():
    p = [torch.zeros(1 << 20, device=DEV)]
    opt = ob.AdamW(p)
    opt.m.fill_(3.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept, copies = delayed_copies(1 << 20, torch.float32)
    ck = opt.checkpoint(stream=side)
    side.synchronize()
    assert torch.equal(ck["m"].cpu(), torch.full((1 << 20,), 3.0))
    assert all(torch.equal(x.cpu(), y) for x, y in zip(copies, kept))
