"""Adapters of the widest rows that are allowed, forward and backward.  Bounds:
tests/test_gpu_adapters.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - GPU tests need a device
    pytest.skip("no CUDA device", allow_module_level=True)

import sparse_mixture_experts_25_b200 as moe  # noqa: E402
from tests.test_gpu_adapters import E  # noqa: E402

WIDEST = 1 << 23


@pytest.mark.parametrize("dtype,r", [("fp32", 24), ("bf16", 72), ("fp32", 128)])
def test_adapter_rows_of_the_largest_width(dtype, r):
    """d_out of 2^23 forward, d_in of 2^23 backward: the sums' columns go in
    more spans than a grid has blocks in y.  33 tokens: the sorted form."""
    N, d, gen = 33, 8, torch.Generator(device="cuda").manual_seed(r)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def normal(*shape, dt=dt):
        return torch.randn(shape, generator=gen, device="cuda").to(dt)

    part = 2.0 ** -21
    scale = torch.ones(1, device="cuda")
    ids = torch.zeros(N, dtype=torch.int32, device="cuda")
    ids[4] = -1
    has = (ids == 0).double()[:, None]
    x, A, B = normal(N, d), normal(1, r, d), normal(1, WIDEST, r)
    ap = moe.adapter_params(N, d, WIDEST, 1, r, dtype=moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32)
    ws = torch.full((moe.moe_adapter_workspace_size(ap),), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.full((N, WIDEST), float("nan"), device="cuda")
    moe.moe_adapter_forward(ap, x, None, A, B, scale, ids, None, y, ws)
    assert moe.moe_adapter_check(ap, ws) == moe.MOE_OK
    u = has * (x.double() @ A[0].double().T)
    mag = x.double().abs() @ A[0].double().abs().T
    eu = has * (((6 * d + 4) * E + part) * mag + part * mag)
    B64 = B[0].double()
    off = (y.double() - u @ B64.T).abs()
    B64.abs_()
    assert bool((off <= eu @ B64.T + ((6 * r + 3) * E + part) * (u.abs() @ B64.T) + 1e-37).all())
    del B, B64, off, y, ws

    # backward with the widths exchanged: dx [N, 2^23] = v A, v from dy [N, 8]
    x, A, B, dy = normal(N, WIDEST), normal(1, r, WIDEST), normal(1, d, r), normal(N, d, dt=torch.float32)
    ap = moe.adapter_params(N, WIDEST, d, 1, r, dtype=ap.dtype)
    ws = torch.full((moe.moe_adapter_backward_workspace_size(ap),), 0xFF, dtype=torch.uint8, device="cuda")
    dx, dA, dB = (torch.full(s, float("nan"), device="cuda") for s in ((N, WIDEST), tuple(A.shape), tuple(B.shape)))
    moe.moe_adapter_backward(ap, x, None, A, B, scale, ids, dy, None, dx, dA, dB, ws)
    assert moe.moe_adapter_check(ap, ws) == moe.MOE_OK
    v = has * (dy.double() @ B[0].double())
    mag = dy.double().abs() @ B[0].double().abs()
    ev = has * (((6 * d + 4) * E + part) * mag + part * mag)
    A64 = A[0].double()
    off = (dx.double() - v @ A64).abs()
    A64.abs_()
    assert bool((off <= ev @ A64 + ((6 * r + 3) * E + part) * (v.abs() @ A64) + 1e-37).all())
    del A64, off
    x64 = x.double()
    off = (dA[0].double() - v.T @ x64).abs()
    x64.abs_()
    assert bool((off <= ev.T @ x64 + ((6 * N + 2) * E + part) * (v.abs().T @ x64) + 1e-37).all())
