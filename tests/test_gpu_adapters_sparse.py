"""Adapter gradients of batches in which few tokens carry an adapter.

The gradients of A and B are summed over ranges of the tokens that have an
adapter, and the call's host side knows only how many tokens there are: with
fewer adapted tokens than ranges, partial sums must come from what this call
wrote and from nothing else.  The workspace is filled with 0xFF (NaN as fp32),
or holds an earlier call's sums.  Bounds: tests/test_gpu_adapters.py.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - GPU tests need a device
    pytest.skip("no CUDA device", allow_module_level=True)

import sparse_mixture_experts_25_b200 as moe  # noqa: E402
from tests.test_gpu_adapters import backward, cuda, make, params, reference, within  # noqa: E402


def sparse_ids(N, n_adapters, adapted, seed):
    """`adapted` tokens at scattered places have an adapter: the last adapter
    about half of them, the others one or two each."""
    rng = np.random.default_rng(seed)
    ids = np.full(N, -1, dtype=np.int32)
    at = rng.permutation(N)[:adapted]
    ids[at] = np.where(np.arange(adapted) % 2 == 0, n_adapters - 1, np.arange(adapted) // 4 % n_adapters)
    return torch.from_numpy(ids)


CASES = [
    # N, d_in, d_out, adapters, r, dtype, W, adapted tokens
    (8, 256, 256, 8, 8, "bf16", False, 2),
    (8, 256, 264, 8, 8, "fp32", False, 3),
    (512, 1024, 1032, 32, 16, "fp32", False, 10),
    (512, 1024, 1024, 32, 16, "bf16", True, 10),
    (2048, 512, 1024, 16, 16, "bf16", False, 21),
    (2048, 1024, 136, 1, 24, "fp32", True, 1),
    (2048, 512, 512, 1024, 8, "bf16", False, 40),
    (8192, 512, 512, 4, 8, "bf16", False, 1),
    (8192, 512, 520, 4, 40, "fp32", False, 12),
    (8192, 264, 512, 4, 128, "bf16", False, 40),
    (8192, 4096, 4096, 4, 8, "bf16", False, 5),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_adapter_gradients_of_few_adapted_tokens(case):
    N, d_in, d_out, a, r, dtype, W, adapted = case
    t = make(N, d_in, d_out, a, r, dtype, "none", W, True)
    t["ids"] = sparse_ids(N, a, adapted, seed=N + adapted)
    want, tol = reference(t, dtype == "bf16")
    got = backward(cuda(t))
    for n in ("dA", "dB", "dx"):
        within(n, got[n], want[n], tol[n])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_replayed_gradient_goes_from_many_adapted_tokens_to_few(dtype):
    """One workspace throughout: a sparse batch must not meet the partial sums
    of the dense one before it."""
    N, d, a, r = 2048, 512, 8, 16
    t = make(N, d, d, a, r, dtype, "mixed", False, True)
    d_ = cuda(t)
    ap = params(d_)
    ws = torch.empty(moe.moe_adapter_backward_workspace_size(ap), dtype=torch.uint8, device="cuda")
    dx, dA, dB = (torch.empty(s, device="cuda") for s in ((N, d), (a, r, d), (a, d, r)))

    def call():
        moe.moe_adapter_backward(ap, d_["x"], None, d_["A"], d_["B"], d_["scale"], d_["ids"], d_["dy"], d_["dx_base"],
                                 dx, dA, dB, ws)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for adapted in (N, 17, 3, 0, 29):
        if adapted < N:
            t["ids"] = sparse_ids(N, a, adapted, seed=adapted)
        d_["ids"].copy_(t["ids"])
        want, tol = reference(t, dtype == "bf16")
        graph.replay()
        torch.cuda.synchronize()
        for n, v in (("dA", dA), ("dB", dB), ("dx", dx)):
            within(f"{n}, {adapted} adapted tokens", v, want[n], tol[n])
