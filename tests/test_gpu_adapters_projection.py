"""W^T dy of a bf16 projection: dy goes in two bf16 parts, and the tensor pipe cuts
off its running sum at every addition."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - GPU tests need a device
    pytest.skip("no CUDA device", allow_module_level=True)

import sparse_mixture_experts_25_b200 as moe  # noqa: E402


@pytest.mark.parametrize("N,d_in,d_out", [(2048, 4096, 4096), (300, 1024, 2056)])
def test_the_small_parts_cost_no_accuracy(N, d_in, d_out):
    """A dy of 16 bits is its two parts exactly, so what is off is cut off from
    running sums.  The small parts are at most 2^-8 of the large ones, and so are
    their sums: added up first, they lose 2^-8 of what the large parts' sums
    lose, and move those by 2^-8.  So dx is as far off as it is for the large
    parts alone, within 2 * 2^-8 and the chance of N d_in cut-off digits: 5%.
    Behind the large parts they would be cut off at the whole sum's size, once
    more for every step of K: about three times as far off."""
    gen = torch.Generator(device="cuda").manual_seed(N)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    x, W = normal(N, d_in).bfloat16(), (normal(d_out, d_in) * d_in ** -0.5).bfloat16()
    A, B = normal(1, 8, d_in).bfloat16(), normal(1, d_out, 8).bfloat16()
    ap = moe.adapter_params(N, d_in, d_out, 1, 8)
    ws = torch.empty(moe.moe_adapter_backward_workspace_size(ap, True), dtype=torch.uint8, device="cuda")
    ids, scale = torch.full((N,), -1, dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda")
    dx, dA, dB = (torch.empty(s, device="cuda") for s in ((N, d_in), tuple(A.shape), tuple(B.shape)))
    dy = normal(N, d_out)
    large = dy.bfloat16().float()
    both = large + (dy - large).bfloat16().float()
    assert torch.equal((both - large).bfloat16().float(), both - large)
    off = []
    for part in (large, both):
        moe.moe_adapter_backward(ap, x, W, A, B, scale, ids, part, None, dx, dA, dB, ws)
        want = part.double() @ W.double()
        off.append(float((dx.double() - want).norm() / want.norm()))
    assert off[1] <= 1.05 * off[0], off
