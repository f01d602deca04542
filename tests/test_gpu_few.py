"""moe_forward_few (the layer for at most 32 tokens) against the layer in 64
bits, on seeded inputs.

Routing records and statistics are held to the same oracle as moe_forward's.
Outputs are compared element by element with the layer evaluated in float64
on the GPU's routing records, within a bound that follows the arithmetic:
  * a sum of n products of 24-bit terms, added in any order, is off by at most
    n 2^-23 times the sum of the products' magnitudes (2^-24 for each rounded
    addition; 2^-23 also covers one that truncates);
  * SiLU moves by at most 1.1 times its argument's error, and its own fp32
    evaluation is off by a few 2^-24 (bounded by 2^-20 of its value);
  * bf16 layers hold h as three bf16 parts: a half step of the third is at most
    2^-24 of h.
"""
import numpy as np
import pytest

import oracle
import seeded_inputs as si
from tests import parity

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - GPU tests need a device
    pytest.skip("no CUDA device", allow_module_level=True)

import sparse_mixture_experts_25_b200 as moe  # noqa: E402

W = si.WORKLOADS
SWITCH, MIXTRAL, QWEN, DEEPSEEK, WDMOE = (W[n] for n in (
    "switch_top1_f32", "mixtral_bf16", "qwen3_skew_bf16", "deepseek_shared_bf16", "wdmoe_decode_bf16"))
CASES = {
    "f32_one": SWITCH.scaled("few_f32_one", N=1, d=64, d_f=96),
    "f32_odd": SWITCH.scaled("few_f32_odd", N=9, d=520, d_f=1032, E=5, k=2, norm=si.NORM_RENORM, c=0.0),
    "f32_all_rows_shared": SWITCH.scaled("few_f32_all", N=32, d=136, d_f=40, E=3, k=3, c=0.0, d_f_shared=1048),
    "f32_capped": SWITCH.scaled("few_f32_capped", N=20, d=72, d_f=48, E=4, k=2, c=0.5, reject_policy=1,
                                norm=si.NORM_RENORM),
    "f32_wide_rows": SWITCH.scaled("few_f32_wide", N=21, d=2056, d_f=72, E=2, k=2, norm=si.NORM_RENORM, c=0.0),
    "f32_two_tiles": SWITCH.scaled("few_f32_tiles", N=3, d=3208, d_f=328, E=6, k=2, norm=si.NORM_RENORM, c=0.0,
                                   d_f_shared=72),
    "f32_long_pieces": SWITCH.scaled("few_f32_long", N=11, d=136, d_f=3400, E=4, k=3, norm=si.NORM_RENORM, c=0.0),
    "narrow_long_pieces": MIXTRAL.scaled("few_narrow_long", N=6, d=96, d_f=6408, E=5, k=3),
    "one_token_wide": MIXTRAL.scaled("few_one_wide", N=1, d=1032, d_f=2056),
    "one_token_one_expert": MIXTRAL.scaled("few_one_expert", N=1, d=8, d_f=8, E=1, k=1),
    "eight": MIXTRAL.scaled("few_eight", N=8, d=512, d_f=264),
    "nine_one_expert": MIXTRAL.scaled("few_nine", N=9, d=320, d_f=136, E=1, k=1),
    "sixteen_odd_experts": MIXTRAL.scaled("few_sixteen", N=16, d=2056, d_f=72, E=34, k=3),
    "full_rows": MIXTRAL.scaled("few_full_rows", N=32, d=264, d_f=520, E=2, k=2),
    "skewed_capped": QWEN.scaled("few_skewed", N=31, d=256, d_f=192, E=129, k=8, c=1.25),
    "many_experts": DEEPSEEK.scaled("few_many", N=17, d=448, d_f=128, E=256, k=8, d_f_shared=24),
    "shared_wider": DEEPSEEK.scaled("few_shared_wide", N=3, d=192, d_f=40, E=16, k=2, d_f_shared=3080),
    "wlr": WDMOE.scaled("few_wlr", N=32, d=512, d_f=640),
    "renorm_reject": QWEN.scaled("few_reject", N=32, d=128, d_f=64, E=8, k=4, c=0.6, reject_policy=1),
    "all_lost": QWEN.scaled("few_all_lost", N=32, d=64, d_f=64, E=2, k=1, c=0.05),
    "thirty_two_of_k": MIXTRAL.scaled("few_k32", N=5, d=64, d_f=64, E=40, k=32),
}


def forward(w, dev, p=None, ws=None, Y=None, stream=None):
    p = p or parity.params_of(w)
    ws = torch.empty(moe.moe_few_workspace_size(p), dtype=torch.uint8, device="cuda") if ws is None else ws
    Y = torch.full((w.N, w.d), float("nan"), device="cuda") if Y is None else Y
    moe.moe_forward_few(p, dev["x"], dev["W_r"], dev.get("b_r"), dev.get("lat"), dev["W_g"], dev["W_u"],
                        dev["W_d"], dev.get("Ws_g"), dev.get("Ws_u"), dev.get("Ws_d"), Y, ws, stream=stream)
    return p, ws, Y


def layer64(w, dev, rec):
    """The layer in float64 on the routing records, and the elementwise bound
    of an fp32 evaluation's error (module docstring)."""
    f = {n: (None if t is None else t.double().cpu()) for n, t in dev.items()}
    wc = torch.from_numpy(oracle.reject_weights(rec["ids"], rec["w"].astype(np.float64), rec["slot"],
                                                w.reject_policy))
    step = 2.0 ** -23
    Y = torch.zeros(w.N, w.d, dtype=torch.float64)
    bound = torch.zeros_like(Y)
    groups = [(f["W_g"][e], f["W_u"][e], f["W_d"][e],
               [(t, float(wc[t, j])) for t in range(w.N) for j in range(w.k)
                if rec["ids"][t, j] == e and rec["slot"][t, j] >= 0]) for e in range(w.E)]
    if w.d_f_shared:
        groups.append((f["Ws_g"], f["Ws_u"], f["Ws_d"], [(t, 1.0) for t in range(w.N)]))
    for Wg, Wu, Wd, rows in groups:
        if not rows:
            continue
        at = torch.tensor([t for t, _ in rows])
        a = torch.tensor([v for _, v in rows], dtype=torch.float64)[:, None]
        x = f["x"][at]
        z, u = x @ Wg.T, x @ Wu.T
        ez, eu = (w.d * step * (x.abs() @ m.abs().T) for m in (Wg, Wu))
        silu = z * torch.sigmoid(z)
        h = silu * u
        eh = 1.1 * ez * (u.abs() + eu) + silu.abs() * eu + (2.0 ** -20 + 2.0 ** -24) * h.abs()
        K = Wd.shape[1]
        y, mag = h @ Wd.T, h.abs() @ Wd.abs().T
        ey = eh @ Wd.abs().T + K * step * mag
        Y[at] += a * y
        # the weighted sum over the groups: k + 1 more additions
        bound[at] += a.abs() * (ey + (w.k + 2) * step * mag)
    return Y, bound


def check(w, dev, inp, ws, p, Y):
    status, stats = moe.moe_get_stats(p, ws)
    assert status == moe.MOE_OK, moe.moe_status_string(status)
    rec = {n: v.cpu().numpy() for n, v in moe.workspace_views(p, ws).items()}
    parity.check_routing(w, inp, rec)
    parity.check_dispatch(w, rec, stats)
    ref, bound = layer64(w, dev, rec)
    off = (Y.double().cpu() - ref).abs()
    assert bool((off <= bound + 1e-37).all()), \
        f"largest error {float(off.max()):.3e}, {float((off / (bound + 1e-37)).max()):.2f} of its bound"
    lost = ~((rec["slot"] >= 0).any(axis=1)) & (w.d_f_shared == 0)
    assert bool((Y.cpu()[torch.from_numpy(lost)] == 0).all())
    return rec, stats


@pytest.mark.parametrize("name", sorted(CASES))
def test_few_matches_the_layer_in_64_bits(name):
    w = CASES[name]
    inp = si.inputs(w)
    dev = {n: parity.to_dev(v) for n, v in inp.items()}
    p, ws, Y = forward(w, dev)
    rec, stats = check(w, dev, inp, ws, p, Y)
    r = oracle.route(inp["x"], inp["W_r"], k=w.k, norm=w.norm, theta=w.theta, b_r=inp.get("b_r"), lat=inp.get("lat"))
    assert abs(stats["aux_balance"] - oracle.aux_balance(r["logits"], rec["ids"], w.E, r["invalid"])) <= 1e-4
    # the same inputs give the same bits, over a workspace and an output of other contents
    Y2 = torch.full_like(Y, float("inf"))
    forward(w, dev, p, torch.full_like(ws, 0xFF), Y2)
    assert torch.equal(Y, Y2)


@pytest.mark.parametrize("w", [
    QWEN.scaled("few_qwen_full", N=3, c=0.0),
    MIXTRAL.scaled("few_mixtral_full", N=2, E=4),
    DEEPSEEK.scaled("few_deepseek_full", N=12, E=64),
], ids=lambda w: w.name)
def test_few_matches_the_layer_of_any_size(w):
    """Widths of the page-shaped layers, random weights made on the device:
    the outputs of moe_forward and moe_forward_few differ by moe_forward's
    rounding of h to bf16 (at most 2^-8 of each term, so 2^-8 of the row's
    largest entry times a few; the layer's own bound is 2e-2)."""
    g = torch.Generator(device="cuda").manual_seed(w.seed)
    dev = {n: None for n in ("b_r", "lat", "Ws_g", "Ws_u", "Ws_d")}
    for n in ("x", "W_r", "W_g", "W_u", "W_d") + (("Ws_g", "Ws_u", "Ws_d") if w.d_f_shared else ()):
        shape = si.shape(w, n)
        dev[n] = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(
            0, 1.0 if n == "x" else shape[-1] ** -0.5, generator=g)
    p, ws, Y = forward(w, dev)
    status, stats = moe.moe_get_stats(p, ws)
    assert status == moe.MOE_OK
    ids = moe.workspace_views(p, ws)["ids"].clone()
    ws2 = torch.empty(moe.moe_workspace_size(p), dtype=torch.uint8, device="cuda")
    Y2 = torch.empty_like(Y)
    moe.moe_forward(p, dev["x"], dev["W_r"], None, None, dev["W_g"], dev["W_u"], dev["W_d"], dev["Ws_g"],
                    dev["Ws_u"], dev["Ws_d"], Y2, ws2)
    assert moe.moe_get_stats(p, ws2)[0] == moe.MOE_OK
    assert torch.equal(ids, moe.workspace_views(p, ws2)["ids"])
    parity.assert_rows_close(Y.double().cpu().numpy(), Y2.double().cpu().numpy(), parity.TOL[w.dtype])


def test_few_empty_batch_and_tokens_that_are_not_finite():
    w = DEEPSEEK.scaled("few_bad", N=6, d=64, d_f=64, E=16, k=2, d_f_shared=32)
    inp = si.inputs(w)
    dev = {n: parity.to_dev(v) for n, v in inp.items()}
    p, ws, Y = forward(w, dev)
    dev["x"][2] = float("nan")
    dev["x"][4, 7] = float("inf")
    p, ws, bad = forward(w, dev)
    status, stats = moe.moe_get_stats(p, ws)
    assert status == moe.MOE_ERR_NONFINITE and stats["nonfinite"] == 2
    assert (moe.workspace_views(p, ws)["ids"][[2, 4]] == -1).all()
    rest = [0, 1, 3, 5]
    assert torch.equal(Y[rest], bad[rest])
    p0 = moe.params(0, 64, 64, 16, 2)
    ws = torch.full((moe.moe_few_workspace_size(p0),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_forward_few(p0, None, None, None, None, None, None, None, None, None, None, None, ws)
    status, stats = moe.moe_get_stats(p0, ws)
    assert status == moe.MOE_OK and stats["requested"] == 0


def test_few_in_a_graph_and_on_two_streams():
    w = QWEN.scaled("few_graph", N=11, d=256, d_f=320, E=16, k=4, c=1.0)
    a, b = ({n: parity.to_dev(v) for n, v in si.inputs(w.scaled(w.name, seed=s)).items()} for s in (1, 2))
    p, ws, Ya = forward(w, a)
    _, _, Yb = forward(w, b)
    # two calls at once, each on a stream and a workspace of its own
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        for s, dev in ((s1, a), (s2, b)):
            with torch.cuda.stream(s):
                outs.append(forward(w, dev)[2])
    torch.cuda.synchronize()
    assert all(torch.equal(y, (Ya, Yb)[i % 2]) for i, y in enumerate(outs))
    # captured, and replayed with another token batch in the same buffers
    x, Y = a["x"].clone(), torch.empty_like(Ya)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(w, dict(a, x=x), p, ws, Y)
    graph.replay()
    assert torch.equal(Y, Ya)
    x.copy_(b["x"])
    graph.replay()
    fresh = forward(w, dict(a, x=x))[2]
    torch.cuda.synchronize()
    assert torch.equal(Y, fresh) and not torch.equal(Y, Ya)


def test_few_takes_hidden_values_at_the_end_of_the_range():
    # h = (181/128)^2 2^127 is finite, but rounds to an infinity in bf16
    p = moe.params(1, 8, 8, 1, 1)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(1, 8, **bf)
    x[0, 0] = 1.0
    W_g, W_u, W_d = (torch.zeros(1, 8, 8, **bf) for _ in range(3))
    W_g[0, 3, 0], W_u[0, 3, 0] = 181 / 128 * 2.0 ** 63, 181 / 128 * 2.0 ** 64
    W_d[0, :, 3] = 2.0 ** -100
    ws = torch.empty(moe.moe_few_workspace_size(p), dtype=torch.uint8, device="cuda")
    Y = torch.empty(1, 8, device="cuda")
    moe.moe_forward_few(p, x, torch.zeros(1, 8, **bf), None, None, W_g, W_u, W_d, None, None, None, Y, ws)
    assert moe.moe_get_stats(p, ws)[0] == moe.MOE_OK
    assert bool((Y == (181 / 128) ** 2 * 2.0 ** 27).all())


def test_few_many_calls_at_once_end():
    """Calls on four streams, each of which needs every SM: none waits for another's half."""
    w = QWEN.scaled("few_at_once", N=32, d=512, d_f=320, E=16, k=4)
    devs = [{n: parity.to_dev(v) for n, v in si.inputs(w.scaled(w.name, seed=s)).items()} for s in range(4)]
    want = [forward(w, dev)[2] for dev in devs]
    bufs = [forward(w, dev) for dev in devs]
    streams = [torch.cuda.Stream() for _ in devs]
    torch.cuda.synchronize()
    for _ in range(25):
        for s, dev, (p, ws, Y) in zip(streams, devs, bufs):
            with torch.cuda.stream(s):
                forward(w, dev, p, ws, Y)
    torch.cuda.synchronize()
    for y, (p, ws, Y) in zip(want, bufs):
        assert moe.moe_get_stats(p, ws)[0] == moe.MOE_OK
        assert torch.equal(y, Y)
