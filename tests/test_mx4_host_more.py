"""Mx4Linear's checks of a weight, without a GPU."""
import pytest
import torch

import communication_compressed_optimizer_momentum_b200 as ob


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
