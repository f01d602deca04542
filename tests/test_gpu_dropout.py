"""moe_dropout_forward and moe_dropout_backward against their definition in 64
bits: the mask has to be the generator's exactly, the values within half a
step of the output's type (bf16 2^-8; the fp32 sum before it and the fp32 type
itself 2^-24, three roundings: the scale, the product, the sum)."""
import numpy as np
import pytest

from tests.philox import kept

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - GPU tests need a device
    pytest.skip("no CUDA device", allow_module_level=True)

import sparse_mixture_experts_25_b200 as moe  # noqa: E402

CASES = [  # N, d, rate, row0, offset
    (1, 8, 0.5, 0, 0),
    (3, 1032, 0.1, 0, 5),
    (257, 520, 0.25, 1000, (1 << 63) + 3),
    (5, 4096, 0.0, 7, 1),
    (64, 64, 0.999, 1 << 40, 2),
    (2, 16, 1 - 2.0 ** -40, 0, 0),
]
SEED = 0xDEADBEEF12345678


def inputs(N, d, dt, seed=0):
    rng = np.random.default_rng(seed)
    Y = torch.from_numpy(rng.standard_normal((N, d))).float()
    return Y, torch.from_numpy(rng.standard_normal((N, d)) * 2).to(dt)


def params(case, dt):
    N, d, rate, row0, offset = case
    return moe.dropout_params(N, d, rate, seed=SEED, offset=offset, row0=row0,
                              dtype=moe.MOE_BF16 if dt == torch.bfloat16 else moe.MOE_F32)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}-{c[2]:.3f}")
def test_dropout_matches_64_bits(case, dt):
    N, d, rate, row0, offset = case
    Y, res = inputs(N, d, dt)
    m = torch.from_numpy(kept(N, d, min(rate, 1 - 2.0 ** -32), SEED, offset, row0))
    dp, half = params(case, dt), torch.finfo(dt).eps / 2
    scaled = torch.where(m, Y.double() / (1 - rate), 0.0)
    for r in (None, res):
        out = torch.full((N, d), float("nan"), dtype=dt, device="cuda")
        moe.moe_dropout_forward(dp, Y.cuda(), None if r is None else r.cuda(), out)
        want = scaled + (0 if r is None else r.double())
        tol = (half + 2.0 ** -24) * want.abs() + 3 * 2.0 ** -24 * scaled.abs()
        assert bool(((out.cpu().double() - want).abs() <= tol).all())
        if r is None:
            assert bool(((out.cpu() != 0) == (m & (Y != 0))).all())
    dY = torch.full((N, d), float("nan"), device="cuda")
    moe.moe_dropout_backward(dp, res.cuda(), dY)
    want = torch.where(m, res.double() / (1 - rate), 0.0)
    assert bool(((dY.cpu().double() - want).abs() <= 3 * 2.0 ** -24 * want.abs()).all())
    # in place: the residual stream, and (fp32) the gradient
    out = res.cuda()
    moe.moe_dropout_forward(dp, Y.cuda(), out, out)
    again = torch.empty_like(out)
    moe.moe_dropout_forward(dp, Y.cuda(), res.cuda(), again)
    assert torch.equal(out, again)
    if dt == torch.float32:
        g = res.cuda()
        moe.moe_dropout_backward(dp, g, g)
        assert torch.equal(g, dY)


def test_dropout_of_a_shard_is_the_whole_batch_s():
    N, d = 37, 264
    Y, res = (t.cuda() for t in inputs(N, d, torch.bfloat16))
    whole = torch.empty_like(res)
    moe.moe_dropout_forward(params((N, d, 0.3, 11, 9), torch.bfloat16), Y, res, whole)
    parts = torch.empty_like(res)
    for lo, hi in ((0, 1), (1, 20), (20, 37)):
        moe.moe_dropout_forward(params((hi - lo, d, 0.3, 11 + lo, 9), torch.bfloat16), Y[lo:hi], res[lo:hi],
                                parts[lo:hi])
    assert torch.equal(whole, parts)


def test_dropout_selects_what_is_not_finite_away():
    N, d = 9, 64
    case = (N, d, 0.5, 0, 3)
    m = torch.from_numpy(kept(N, d, 0.5, SEED, 3, 0))
    Y = torch.full((N, d), float("inf"))
    Y[::2] = float("nan")
    out = torch.empty(N, d, device="cuda")
    moe.moe_dropout_forward(params(case, torch.float32), Y.cuda(), None, out)
    assert bool((out.cpu()[~m] == 0).all()) and not bool(out.cpu()[m].isfinite().any())


def test_dropout_share_of_kept_elements():
    # 2^22 draws: within five standard deviations of the rate
    N, d, rate = 1024, 4096, 0.1
    out = torch.empty(N, d, device="cuda")
    moe.moe_dropout_forward(params((N, d, rate, 0, 77), torch.float32), torch.ones(N, d, device="cuda"), None, out)
    n = N * d
    assert abs(float((out == 0).double().mean()) - rate) <= 5 * (rate * (1 - rate) / n) ** 0.5


def test_dropout_in_a_graph_draws_by_the_step():
    N, d = 65, 128
    Y, res = (t.cuda() for t in inputs(N, d, torch.float32))
    out, dY = torch.empty_like(res), torch.empty_like(res)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    dp = params((N, d, 0.25, 0, 40), torch.float32)
    graph = torch.cuda.CUDAGraph()
    moe.moe_dropout_forward(dp, Y, res, out, step=step)
    with torch.cuda.graph(graph):
        moe.moe_dropout_forward(dp, Y, res, out, step=step)
        moe.moe_dropout_backward(dp, res, dY, step=step)
        step.add_(1)
    for i in range(3):
        graph.replay()
        m = torch.from_numpy(kept(N, d, 0.25, SEED, 40 + i, 0))
        assert torch.equal(dY.cpu() != 0, m & (res.cpu() != 0))
        fresh = torch.empty_like(out)
        moe.moe_dropout_forward(params((N, d, 0.25, 0, 40 + i), torch.float32), Y, res, fresh)
        assert torch.equal(out, fresh)
