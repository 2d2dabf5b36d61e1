"""Mx4Linear without a GPU: the checks of a weight, and the seeds of its backward pass."""
import numpy as np
import pytest
import torch

import communication_compressed_optimizer_momentum_b200 as ob
import mx4_reference as ref


def linear(outer, inner):
    """A layer whose matrix in 4 bits lies on the CPU: enough for the checks."""
    layer = ob.Mx4Linear.__new__(ob.Mx4Linear)
    layer.outer, layer.inner = outer, inner
    layer.w, layer.wt = ob.Mx4.empty(outer, inner, device="cpu"), None
    return layer


@pytest.mark.parametrize("weight,error,why", [
    (torch.zeros(40, 40, dtype=torch.float16), TypeError, "float32 or bfloat16"),
    (torch.zeros(40, 40, dtype=torch.float64), TypeError, "float32 or bfloat16"),
    (torch.zeros(40, 40, dtype=torch.int32), TypeError, "float32 or bfloat16"),
    (torch.zeros(40, 40).t(), ValueError, None),
    (torch.zeros(40, 41).t()[:40], ValueError, "consecutive columns"),
    (torch.zeros(40, 80)[:, ::2], ValueError, "consecutive columns"),
    (torch.zeros(40).expand(40, 40), ValueError, "rows of its own"),
    (torch.zeros(2000).as_strided((40, 40), (39, 1)), ValueError, "rows of its own"),
    (torch.zeros(40, 41), ValueError, "40 x 40"),
    ([0.0], ValueError, "40 x 40"),
])
def test_a_weight_that_update_would_refuse(weight, error, why):
    with pytest.raises(error, match=why):
        linear(40, 40).check_weight(weight)


def test_weights_that_update_takes():
    for w in (torch.zeros(40, 40), torch.zeros(40, 40, dtype=torch.bfloat16),
              torch.zeros(42, 50)[1:41, 3:43]):
        linear(40, 40).check_weight(w)
    linear(1, 40).check_weight(torch.zeros(40).expand(1, 40))        # one row: its stride means nothing
    linear(40, 1).check_weight(torch.zeros(40, 5)[:, 2:3])
    linear(40, 0).check_weight(torch.zeros(40, 0))


def test_seeds_two_apart_share_no_bits():
    """The transposed form takes the bits of seed + 1, and so does the row form of the next seed: of seeds
    two apart, as layers and steps are to take them, no two forms have the same key."""
    place = np.arange(4096)
    layers, steps = 3, 4
    seeds = [2 * (step * layers + layer) for step in range(steps) for layer in range(layers)]
    bits = [ref.random16(place, s + form) for s in seeds for form in (0, 1)]
    assert len({b.tobytes() for b in bits}) == 2 * len(seeds)
    for i, a in enumerate(bits):                       # equal by chance only: 1 in 65536
        assert all((a == b).sum() < 8 for b in bits[:i])


def test_matrices_whose_bytes_64_bits_do_not_count():
    """Refused before their ranges are compared: (rows - 1) * ld * 4 would come out as anything."""
    from communication_compressed_optimizer_momentum_b200 import _abi, build
    build.build()
    lib = _abi.lib()
    x, codes, scales = 1 << 40, 1 << 50, 1 << 52
    for rows, ld in ((1 << 30, 1 << 40), (1 << 25, 1 << 40), ((1 << 20) + 1, 1 << 40)):
        for rc in (lib.onebit_mx4_quantize(rows, 70, x, 0, ld, codes, scales, None, None, 0, 1, None, 0, None),
                   lib.onebit_mx4_quantize(rows, 70, x, 1, 70, codes, scales, None, None, 0, 1, 1 << 55, ld,
                                           None),
                   lib.onebit_mx4_dequantize(rows, 70, codes, scales, x, 1, ld, None),
                   lib.onebit_mx4_matmul(rows, 70, 64, codes, scales, 1 << 54, 1 << 55, x, 0, ld, 0, None),
                   lib.onebit_mx4_linear(rows, 70, 64, x, 0, ld, 1 << 54, 1 << 55, codes, scales, None, None,
                                         1 << 56, 0, 70, None)):
            assert rc == -1 and "row stride" in lib.onebit_last_error().decode()
