"""More of AdamW without a GPU: lengths beyond 64 bits, and parameters that no step would take."""
import pytest
import torch

import communication_compressed_optimizer_momentum_b200 as ob


@pytest.mark.parametrize("n", [1 << 63, (1 << 64) - 1, 1 << 64, (1 << 64) + 300, -(1 << 63) - 1,
                               -(1 << 64) + 5])
def test_layout_refuses_lengths_beyond_64_bits(n):
    with pytest.raises(ob.OneBitError, match="size"):
        ob.onebit_adamw_layout([5, n])


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int32, torch.complex64])
@pytest.mark.parametrize("state", ["q8", "f32"])
def test_an_optimizer_refuses_parameters_that_its_step_would(dtype, state):
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ob.AdamW([torch.zeros(8, dtype=dtype)], state=state)
    with pytest.raises(TypeError, match="list of tensors"):
        ob.AdamW([1.0], state=state)
