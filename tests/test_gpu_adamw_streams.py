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
