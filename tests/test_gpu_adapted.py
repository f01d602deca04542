"""The few-token layer, the adapters and the dropout as they run together
(sparse_mixture_experts_25_b200.adapted), against the composition of the layer's
oracle with the adapters and the mask in 64 bits.

Tolerances are the layer's own (tests/parity.py and tests/test_gpu_backward.py):
what the adapters and the dropout add is far more exact than they are."""
import numpy as np
import pytest

import oracle
import seeded_inputs as si
from tests import parity
from tests.philox import kept

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - GPU tests need a device
    pytest.skip("no CUDA device", allow_module_level=True)

import sparse_mixture_experts_25_b200 as moe  # noqa: E402
from sparse_mixture_experts_25_b200.adapted import WEIGHTS, AdaptedLayer  # noqa: E402

W = si.WORKLOADS
CASES = {
    "bf16": W["mixtral_bf16"].scaled("adapted_bf16", N=300, d=320, d_f=384),
    "shared": W["deepseek_shared_bf16"].scaled("adapted_shared", N=130, d=192, d_f=128, E=16, k=4, d_f_shared=64),
    "f32_capped": W["switch_top1_f32"].scaled("adapted_f32", N=200, d=72, d_f=96, c=0.9),
    "few": W["qwen3_skew_bf16"].scaled("adapted_few", N=11, d=256, d_f=192, E=16, k=2),
    "few_f32": W["switch_top1_f32"].scaled("adapted_few_f32", N=3, d=264, d_f=72, E=4, k=2, c=0.0),
}
RATE, SEED, ADAPTERS, RANK = 0.2, 99, 5, 16


def build(w, rate):
    inp = si.inputs(w)
    dev = {n: parity.to_dev(v) for n, v in inp.items()}
    rng = np.random.default_rng(w.N)
    dt = dev["x"].dtype
    A = torch.from_numpy(rng.standard_normal((ADAPTERS, RANK, w.d)) * w.d ** -0.5).to(dt)
    B = torch.from_numpy(rng.standard_normal((ADAPTERS, w.d, RANK)) * RANK ** -0.5).to(dt)
    scale = torch.from_numpy(rng.uniform(0.5, 2, ADAPTERS)).float()
    ids = torch.from_numpy(rng.integers(-1, ADAPTERS, w.N)).int()
    residual = torch.from_numpy(rng.standard_normal((w.N, w.d))).to(dt)
    layer = AdaptedLayer(parity.params_of(w), {n: dev.get(n) for n in WEIGHTS}, A.cuda(), B.cuda(), scale.cuda(),
                         rate=rate, seed=SEED)
    return inp, dev, layer, A.double(), B.double(), scale.double(), ids, residual


def records(layer):
    return {n: v.cpu().numpy() for n, v in moe.workspace_views(layer.p, layer.ws).items()}


def layer_rows(w, inp, rec):
    wc = oracle.reject_weights(rec["ids"], rec["w"].astype(np.float64), rec["slot"], w.reject_policy)
    Ws = (inp["Ws_g"], inp["Ws_u"], inp["Ws_d"]) if w.d_f_shared else None
    return torch.from_numpy(oracle.forward_rows(inp["x"], rec["ids"], wc, rec["slot"], np.arange(w.N), inp["W_g"],
                                                inp["W_u"], inp["W_d"], Ws=Ws))


def low_rank(x, A, B, scale, ids):
    y = torch.zeros(len(ids), B.shape[1], dtype=torch.float64)
    for a in range(len(scale)):
        at = ids == a
        y[at] = scale[a] * (x[at] @ A[a].T) @ B[a].T
    return y


@pytest.mark.parametrize("name", sorted(CASES))
def test_training_step_of_the_adapted_layer(name):
    w = CASES[name]
    inp, dev, layer, A, B, scale, ids, residual = build(w, RATE)
    out = layer.forward(dev["x"], ids.cuda(), residual.cuda(), training=True, offset=4, row0=16)
    layer.check()
    rec = records(layer)
    x = dev["x"].double().cpu()
    m = torch.from_numpy(kept(w.N, w.d, RATE, SEED, 4, 16))
    Y = layer_rows(w, inp, rec) + low_rank(x, A, B, scale, ids)
    want = residual.double() + torch.where(m, Y / (1 - RATE), 0.0)
    parity.assert_rows_close(out.double().cpu().numpy(), want.numpy(), parity.TOL[w.dtype])

    rng = np.random.default_rng(7)
    dout = torch.from_numpy(rng.standard_normal((w.N, w.d))).to(out.dtype)
    g = layer.backward(dout.cuda(), aux_coef=0.2)
    layer.check()
    dY = torch.where(m, dout.double() / (1 - RATE), 0.0)
    Ws = (inp["Ws_g"], inp["Ws_u"], inp["Ws_d"]) if w.d_f_shared else None
    ref = oracle.backward(inp["x"], inp["W_r"], inp["W_g"], inp["W_u"], inp["W_d"], dY.numpy().astype(np.float32),
                          rec["ids"], rec["w"], rec["slot"], norm=w.norm, reject_policy=w.reject_policy,
                          b_r=inp.get("b_r"), Ws=Ws, aux_coef=0.2)
    ref["dA"], ref["dB"] = np.zeros(A.shape), np.zeros(B.shape)
    dx = np.asarray(ref["dx"])
    for a in range(ADAPTERS):
        at = (ids == a).numpy()
        v, u = float(scale[a]) * (dY[at] @ B[a]), float(scale[a]) * (x[at] @ A[a].T)
        dx[at] += (v @ A[a]).numpy()
        ref["dA"][a], ref["dB"][a] = (v.T @ x[at]).numpy(), (dY[at].T @ u).numpy()
    assert set(g) >= {"dx", "dA", "dB", "dW_r", "dW_g", "dW_u", "dW_d"}
    for n, t in g.items():
        tol = 1e-4 if w.dtype == si.DT_F32 else (2e-3 if n in ("dW_r", "db_r") else 5e-3)
        assert parity.rel_err(t.double().cpu().numpy(), np.asarray(ref[n])) <= tol, n
    with pytest.raises(ValueError):
        layer.forward(dev["x"], ids.cuda(), residual.cuda())
        layer.backward(dout.cuda())


@pytest.mark.parametrize("name", sorted(CASES))
def test_serving_step_of_the_adapted_layer(name):
    """Nothing is dropped, whatever the rate; up to 32 tokens take the few-token form."""
    w = CASES[name]
    inp, dev, layer, A, B, scale, ids, residual = build(w, RATE)
    assert layer.few == (w.N <= 32)
    out = layer.forward(dev["x"], ids.cuda(), residual.cuda())
    layer.check()
    want = residual.double() + layer_rows(w, inp, records(layer)) + low_rank(dev["x"].double().cpu(), A, B, scale, ids)
    parity.assert_rows_close(out.double().cpu().numpy(), want.numpy(), parity.TOL[w.dtype])
    # a step that is captured and replayed on other tokens of other requests
    x, i, res = dev["x"].clone(), ids.cuda(), residual.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.forward(x, i, res)
    x.copy_(dev["x"].flip(0))
    i.copy_(ids.flip(0))
    res.copy_(residual.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    if w.c <= 0:  # without a capacity limit a token's output does not hang on its place
        parity.assert_rows_close(got.flip(0).double().cpu().numpy(), want.numpy(), parity.TOL[w.dtype])


def test_adapted_layer_reports_what_a_step_met():
    inp, dev, layer, A, B, scale, ids, residual = build(CASES["few"], 0.0)
    ids[2] = ADAPTERS
    layer.forward(dev["x"], ids.cuda(), residual.cuda())
    with pytest.raises(moe.MoEError, match="adapters"):
        layer.check()
    dev["x"][1, 0] = float("nan")
    layer.forward(dev["x"], ids.cuda(), residual.cuda())
    with pytest.raises(moe.MoEError, match="layer"):
        layer.check()
