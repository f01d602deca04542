"""Adapter gradients through a bf16 projection with a dy at the end of fp32's
range, or past it.  Bounds: tests/test_gpu_adapters.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - GPU tests need a device
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.test_gpu_adapters import backward, cuda, forward, make, reference, within  # noqa: E402


@pytest.mark.parametrize("N", [20, 300, 1500])
def test_a_projection_takes_the_largest_finite_gradients(N):
    """dy within half a bf16 step of the end of the range: finite results stay
    finite, on both signs, and neighbours in the same 16 bytes keep theirs."""
    t = make(N, 136, 264, 3, 16, "bf16", "mixed", True, False)
    top = torch.finfo(torch.float32).max
    bad = 11
    t["dy"][bad, 5], t["dy"][bad, 6], t["dy"][bad, 8] = top, 0.5, -top
    t["dy"][bad + 1, 5] = 2.0 ** 127 * (2 - 2.0 ** -8)  # the first value that rounds past the end
    # factors that keep every result inside the range
    t["W"][5] *= 1e-3
    t["W"][8] *= 1e-3
    t["B"][:, 5] *= 1e-3
    t["B"][:, 8] *= 1e-3
    t["x"][bad:bad + 2] *= 1e-3
    t["scale"][:] = 1e-3
    want, tol = reference(t, True)
    assert all(bool((want[n].abs() < 3e38).all()) for n in ("dx", "dA", "dB"))
    got = backward(cuda(t))
    for n in ("dx", "dA", "dB"):
        within(n, got[n], want[n], tol[n])


def test_a_projection_keeps_what_is_not_finite_in_its_token():
    t = make(300, 136, 264, 3, 16, "bf16", "none", True, False)
    clean = backward(cuda(t))["dx"]
    t["dy"][7, 4], t["dy"][9, 5], t["dy"][10, 5] = float("inf"), float("nan"), float("-inf")
    dx = backward(cuda(t))["dx"]
    rest = [i for i in range(300) if i not in (7, 9, 10)]
    assert torch.equal(dx[rest], clean[rest])
    assert not dx[[7, 9, 10]].isfinite().any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [3, 300])
def test_the_scale_meets_the_whole_sum(N, dtype):
    """u = scale A x of parts of K that nearly cancel: each of them times the scale
    is past the end of the range, their sum is not.  All values are powers of two
    but one, so that the sums are exact in any order, in fp32 too."""
    K, r, d_out = 4096, 8, 64
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.full((N, K), 2.0 ** 10)
    x[:, K // 2:] *= -1
    x[:, 0] += torch.arange(N) % 7 * 2.0 ** 3  # the sum: 2^13 times 0 to 6, in 8 significant bits of x
    A, B = torch.full((1, r, K), 2.0 ** 10), torch.full((1, d_out, r), 2.0 ** -60)
    scale = torch.tensor([2.0 ** 100])
    t = dict(x=x.to(dt), W=None, A=A.to(dt), B=B.to(dt), scale=scale, ids=torch.zeros(N, dtype=torch.int32), base=None)
    assert bool(((x.abs()[:, :256] * A[0, 0, :256]).sum(1) * scale > torch.finfo(torch.float32).max).all())
    u = scale.double() * (t["x"].double() @ A[0].double().T)
    want = u @ B[0].double().T
    y = forward(cuda(t)).double().cpu()
    assert torch.equal(y, want)
