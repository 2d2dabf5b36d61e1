"""A product whose waits give up: it says so, leaves nothing behind and the next one is right."""
import ctypes
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def child():
    """The flag stays set for as long as a process has the device: in a process of its own. The waits'
    limit is set to 1 ns (they then take about 2 ms, the polls before and behind the first look at the
    clock), and the common axis is so long that a tile takes more: the warps that write out give up while
    loads and products go on. Nothing on the device waits for what does not come."""
    import torch

    import communication_compressed_optimizer_momentum_b200 as ob
    from communication_compressed_optimizer_momentum_b200 import _abi
    from test_gpu_mx4_more import held, tiles

    limit = _abi.lib().onebit_internal_mx4_wait
    limit.restype = None

    def long(rows, k):
        codes, scales = ob.onebit_mx4_layout(rows, k)
        return ob.Mx4(torch.zeros(codes, dtype=torch.uint8, device="cuda"),
                      torch.full((scales,), 127, dtype=torch.uint8, device="cuda"), rows, k)

    def right():
        for m, n, k in ((600, 5000, 2000), (2100, 2000, 3000), (16, 2000, 5000), (200, 3000, 1000)):
            (qa, a), (qb, b) = held(m, k, 1), held(n, k, 2)
            for dtype in (torch.float32, torch.bfloat16):
                assert torch.equal(ob.onebit_mx4_matmul(qa, qb, dtype=dtype), (a @ b.t()).to(dtype))

    right()
    assert ob.onebit_mx4_status() == 0
    # pairs of blocks, one tile each; then a cluster that shares a tile
    for m, n, k, want in ((2100, 2000, 6 << 20, (256, 1)), (32, 128, 1 << 26, (32, 8))):
        assert tiles(m, n, k, torch.float32) == want
        a = long(max(m, n), k)
        b = ob.Mx4(a.codes, a.scales, n, k)
        a.rows = m
        out = torch.full((m, n), 3.0, device="cuda")
        limit(ctypes.c_uint64(1))
        ob.onebit_mx4_matmul(a, b, out=out)
        limit(ctypes.c_uint64(0))
        torch.cuda.synchronize()
        assert ob.onebit_mx4_status() == 1
        assert want[1] > 1 or bool((out == 3.0).any())      # a tile that was not written
        del a, b, out
        right()


def test_a_product_that_gives_up():
    env = dict(os.environ, PYTHONPATH=os.pathsep.join(
        [ROOT, os.path.join(ROOT, "tests"), os.environ.get("PYTHONPATH", "")]))
    p = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, capture_output=True,
                       text=True, timeout=120)
    assert p.returncode == 0, p.stdout + p.stderr


if __name__ == "__main__":
    child()
