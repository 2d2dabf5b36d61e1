"""More of AdamW without a GPU: lengths beyond 64 bits."""
import pytest

import communication_compressed_optimizer_momentum_b200 as ob


@pytest.mark.parametrize("n", [1 << 63, (1 << 64) - 1, 1 << 64, (1 << 64) + 300, -(1 << 63) - 1,
                               -(1 << 64) + 5])
def test_layout_refuses_lengths_beyond_64_bits(n):
    with pytest.raises(ob.OneBitError, match="size"):
        ob.onebit_adamw_layout([5, n])
