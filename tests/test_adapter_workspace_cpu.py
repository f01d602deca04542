"""What the adapters' backward workspace holds: rows of u and v and partial sums
of ranges of tokens, not another copy of every adapter's gradients."""
import pytest

import sparse_mixture_experts_25_b200 as moe

pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [moe.MOE_BF16, moe.MOE_F32])
@pytest.mark.parametrize("with_W", [False, True])
def test_adapter_backward_workspace_does_not_grow_with_the_adapters(dtype, with_W):
    few, many = (moe.moe_adapter_backward_workspace_size(moe.adapter_params(4096, 4096, 4096, a, 64, dtype=dtype), with_W)
                 for a in (8, 1024))
    # an adapter's place in the sort (4 bytes) and a tile's record (16 bytes), each region to 256 bytes
    assert many - few <= (1024 - 8) * (4 + 16) + 2 * 256
