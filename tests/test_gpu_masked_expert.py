"""A token one of whose scores is not finite while the others are (an expert
masked by a bias of -inf): it has no paths, is counted, and nothing is read for
an expert that was not chosen -- under weight-latency-ratio pruning the first
token's latencies begin where the caller's buffer begins."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - GPU tests need a device
    pytest.skip("no CUDA device", allow_module_level=True)

import seeded_inputs as si  # noqa: E402
import sparse_mixture_experts_25_b200 as moe  # noqa: E402
from tests import parity  # noqa: E402

NORMS = {"renorm": moe.MOE_NORM_RENORM, "fullprob": moe.MOE_NORM_FULLPROB, "wlr": moe.MOE_NORM_WLR}


@pytest.mark.parametrize("norm", sorted(NORMS))
@pytest.mark.parametrize("E", [5, 40, 130])
@pytest.mark.parametrize("few", [False, True], ids=["batch", "few"])
def test_a_masked_expert_takes_all_paths_of_its_tokens(few, E, norm):
    N, d, d_f, k = 7, 64, 72, 3
    p = moe.params(N=N, d=d, d_f=d_f, E_r=E, k=k, norm=NORMS[norm], theta=0.1, dtype=moe.MOE_F32)
    gen = torch.Generator(device="cuda").manual_seed(E)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    x, W_r, W_g, W_u, W_d = normal(N, d), normal(E, d), normal(E, d_f, d), normal(E, d_f, d), normal(E, d, d_f)
    b_r, lat = torch.zeros(E, device="cuda"), torch.rand(N, E, generator=gen, device="cuda") + 0.5
    size, call = (moe.moe_few_workspace_size, moe.moe_forward_few) if few else (moe.moe_workspace_size, moe.moe_forward)
    ws = torch.full((size(p),), 0xFF, dtype=torch.uint8, device="cuda")
    Y = torch.full((N, d), float("nan"), device="cuda")
    lat_arg = lat if norm == "wlr" else None

    def run():
        call(p, x, W_r, b_r, lat_arg, W_g, W_u, W_d, None, None, None, Y, ws)
        status, stats = moe.moe_get_stats(p, ws)
        rec = {n: v.clone() for n, v in moe.workspace_views(p, ws).items() if n in ("ids", "w")}
        return status, stats, rec, Y.clone()

    status, _, clean, Y_clean = run()
    assert status == moe.MOE_OK and bool((clean["ids"][:, 0] >= 0).all())
    # every token's score of the last expert
    b_r[E - 1] = float("-inf")
    status, stats, rec, got = run()
    assert status == moe.MOE_ERR_NONFINITE and stats["nonfinite"] == N and stats["requested"] == 0
    assert bool((rec["ids"] == -1).all()) and not rec["w"].any() and not got.any()
    # one token's scores only, the first one's: the others keep their paths
    b_r[E - 1] = 0
    x[0, 3] = float("nan")
    status, stats, rec, got = run()
    assert status == moe.MOE_ERR_NONFINITE and stats["nonfinite"] == 1
    assert bool((rec["ids"][0] == -1).all()) and not rec["w"][0].any()
    assert torch.equal(rec["ids"][1:], clean["ids"][1:])
    # the same function of the same rows, but not the same bits: the batch layer adds a token's
    # paths in any order, and both cut their sums by the rows that an expert has.  Each output is
    # within parity.TOL of the largest exact one, so they are within TOL + TOL, relative to a
    # largest output that is itself TOL off
    tol = parity.TOL[si.DT_F32]
    parity.assert_rows_close(got[1:].double().cpu().numpy(), Y_clean[1:].double().cpu().numpy(), 2 * tol / (1 - tol))
