"""moe_adapter_forward and moe_adapter_backward against their definition in 64
bits, element by element.

Bounds, with e = 2^-23 for a rounded or truncated addition:
  * a sum of n products is off by at most n e times the sum of the products'
    magnitudes;
  * an operand held as three bf16 parts is off by at most 2^-24 of its value (a
    half step is 2^-8, three times); the products of parts that are left out
    (second by third and beyond) are below 2^-22 of the whole.  The dy of a
    bf16 projection is held as two parts: 2^-16;
  * an error in u or v carries on through the magnitudes of what multiplies it.
"""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - GPU tests need a device
    pytest.skip("no CUDA device", allow_module_level=True)

import sparse_mixture_experts_25_b200 as moe  # noqa: E402

E = 2.0 ** -23


def ids_of(kind, N, a, rng):
    if kind == "none":
        ids = np.full(N, -1)
    elif kind == "one":
        ids = np.full(N, a - 1)
    elif kind == "runs":
        ids = np.sort(rng.integers(-1, a, N))[::-1].copy()
    elif kind == "own":  # every token its own, as far as they go
        ids = np.arange(N) % a
    else:
        ids = rng.integers(-1, a, N)
    return torch.from_numpy(ids.astype(np.int32))


def make(N, d_in, d_out, a, r, dtype, kind, W, base, seed=0):
    rng = np.random.default_rng(1000 + seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def normal(*shape, std=1.0, dt=dt):
        return torch.from_numpy(rng.standard_normal(shape) * std).to(dt)

    t = {"x": normal(N, d_in), "W": normal(d_out, d_in, std=d_in ** -0.5) if W else None,
         "A": normal(a, r, d_in, std=d_in ** -0.5), "B": normal(a, d_out, r, std=r ** -0.5),
         "scale": torch.from_numpy(rng.uniform(0.5, 1.5, a)).float(), "ids": ids_of(kind, N, a, rng),
         "dy": normal(N, d_out, dt=torch.float32)}
    t["base"] = normal(N, d_out, dt=torch.float32) if base else None
    t["dx_base"] = normal(N, d_in, dt=torch.float32) if base else None
    return t


def reference(t, bf16):
    """The definition in float64 and the elementwise bounds."""
    f = {n: (v.double() if v is not None and n != "ids" else v) for n, v in t.items()}
    N, d_in = t["x"].shape
    d_out, a = t["B"].shape[1], t["A"].shape[0]
    part = 2.0 ** -21  # fp32 operands' parts and the products left out
    split = 2.0 ** -16 if bf16 else 0.0  # dy in front of W
    out = {"y": torch.zeros(N, d_out, dtype=torch.float64), "dx": torch.zeros(N, d_in, dtype=torch.float64),
           "dA": torch.zeros_like(f["A"]), "dB": torch.zeros_like(f["B"])}
    tol = {n: torch.zeros_like(v) for n, v in out.items()}
    for n, b in (("y", "base"), ("dx", "dx_base")):
        if f[b] is not None:
            out[n] += f[b]
            tol[n] += 2 * E * f[b].abs()
    if f["W"] is not None:
        out["y"] += f["x"] @ f["W"].T
        tol["y"] += (d_in + 2) * E * (f["x"].abs() @ f["W"].abs().T)
        out["dx"] += f["dy"] @ f["W"]
        tol["dx"] += ((2 * d_out + 2) * E + split) * (f["dy"].abs() @ f["W"].abs())
    for i in range(a):
        at = torch.nonzero(t["ids"] == i).reshape(-1)
        if not len(at):
            continue
        A, B, s, x, dy = f["A"][i], f["B"][i], f["scale"][i], f["x"][at], f["dy"][at]
        r, n = A.shape[0], len(at)
        u, v = s * (x @ A.T), s * (dy @ B)
        eu = s * (((1 if bf16 else 6) * d_in + 4) * E + (0 if bf16 else part)) * (x.abs() @ A.abs().T) + part * u.abs()
        ev = s * ((6 * d_out + 4) * E + part) * (dy.abs() @ B.abs()) + part * v.abs()
        out["y"][at] += u @ B.T
        tol["y"][at] += eu @ B.abs().T + ((6 * r + 3) * E + part) * (u.abs() @ B.abs().T)
        out["dx"][at] += v @ A
        tol["dx"][at] += ev @ A.abs() + ((6 * r + 3) * E + part) * (v.abs() @ A.abs())
        out["dA"][i] = v.T @ x
        tol["dA"][i] = ev.T @ x.abs() + ((6 * n + 2) * E + part) * (v.abs().T @ x.abs())
        out["dB"][i] = dy.T @ u
        tol["dB"][i] = dy.abs().T @ eu + ((6 * n + 2) * E + part) * (dy.abs().T @ u.abs())
    return out, tol


def params(t):
    a, r, d_in = t["A"].shape
    return moe.adapter_params(len(t["ids"]), d_in, t["B"].shape[1], a, r,
                              dtype=moe.MOE_BF16 if t["A"].dtype == torch.bfloat16 else moe.MOE_F32)


def cuda(t):
    return {n: None if v is None else v.cuda() for n, v in t.items()}


def workspace(size, ap, W, fill=0xFF):
    return torch.full((size(ap, W is not None),), fill, dtype=torch.uint8, device="cuda")


def forward(d, in_place=False, ws=None):
    ap = params(d)
    ws = workspace(moe.moe_adapter_workspace_size, ap, d["W"]) if ws is None else ws
    y = d["base"].clone() if in_place else torch.full((ap.N, ap.d_out), float("nan"), device="cuda")
    moe.moe_adapter_forward(ap, d["x"], d["W"], d["A"], d["B"], d["scale"], d["ids"], y if in_place else d["base"],
                            y, ws)
    assert moe.moe_adapter_check(ap, ws) == moe.MOE_OK
    return y


def backward(d, in_place=False):
    ap = params(d)
    ws = workspace(moe.moe_adapter_backward_workspace_size, ap, d["W"])
    nan = {n: torch.full(s, float("nan"), device="cuda") for n, s in (
        ("dx", (ap.N, ap.d_in)), ("dA", tuple(d["A"].shape)), ("dB", tuple(d["B"].shape)))}
    if in_place:
        nan["dx"] = d["dx_base"].clone()
    moe.moe_adapter_backward(ap, d["x"], d["W"], d["A"], d["B"], d["scale"], d["ids"], d["dy"],
                             nan["dx"] if in_place else d["dx_base"], nan["dx"], nan["dA"], nan["dB"], ws)
    assert moe.moe_adapter_check(ap, ws) == moe.MOE_OK
    return nan


def within(name, got, want, tol):
    off = (got.double().cpu() - want).abs()
    assert bool((off <= tol + 1e-37).all()), \
        f"{name}: largest error {float(off.max()):.3e}, {float((off / (tol + 1e-37)).max()):.2f} of its bound"


CASES = [
    # N, d_in, d_out, adapters, r, dtype, ids, W, base
    (1, 64, 72, 1, 8, "bf16", "one", False, False),
    (1, 4096, 1032, 3, 16, "bf16", "mixed", True, True),
    (5, 520, 264, 17, 24, "fp32", "own", False, True),
    (32, 2056, 520, 70, 128, "bf16", "own", False, True),
    (32, 1000, 136, 4, 40, "fp32", "mixed", True, False),
    (33, 136, 8, 5, 8, "bf16", "mixed", False, True),
    (64, 8, 264, 2, 64, "fp32", "one", False, False),
    (65, 1096, 200, 1, 16, "bf16", "one", True, True),
    (200, 328, 392, 70, 16, "bf16", "own", False, True),
    (257, 2048, 1024, 3, 32, "bf16", "none", False, True),
    (257, 264, 136, 3, 32, "fp32", "none", False, False),
    (300, 520, 648, 7, 40, "fp32", "mixed", False, True),
    (300, 1032, 264, 7, 40, "bf16", "mixed", True, False),
    (517, 4104, 72, 9, 64, "bf16", "runs", False, False),
    (517, 192, 1160, 3, 128, "fp32", "runs", True, True),
    (700, 200, 4104, 1024, 8, "bf16", "mixed", False, True),
    (1111, 768, 520, 2, 128, "bf16", "runs", True, True),
]
IDS = ["-".join(str(v) for v in c) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_adapter_forward_matches_64_bits(case):
    t = make(*case)
    want, tol = reference(t, case[5] == "bf16")
    d = cuda(t)
    y = forward(d)
    within("y", y, want["y"], tol["y"])
    if d["base"] is not None and d["W"] is None:
        assert torch.equal(forward(d, in_place=True), y)
    if d["W"] is None:
        assert torch.equal(forward(d), y)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_adapter_gradients_match_64_bits(case):
    t = make(*case)
    want, tol = reference(t, case[5] == "bf16")
    d = cuda(t)
    got = backward(d)
    for n in ("dx", "dA", "dB"):
        within(n, got[n], want[n], tol[n])
    if d["W"] is None:
        again = backward(d, in_place=d["dx_base"] is not None)
        assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("N", [9, 150])
def test_adapter_gradients_are_the_slopes_of_the_forward(N):
    """y is linear in each of x, A and B, so a central difference of the loss
    <dy, y> along any direction is its slope; fp32, differences of sums of
    about N d_out terms of size 1."""
    t = make(N, 72, 40, 3, 16, "fp32", "mixed", True, True, seed=N)
    d = cuda(t)
    g = backward(dict(d, dx_base=None))
    for n, grad in (("x", "dx"), ("A", "dA"), ("B", "dB")):
        gen = torch.Generator(device="cuda").manual_seed(N)
        step = torch.randn(d[n].shape, generator=gen, device="cuda")
        loss = [float((d["dy"].double() * forward(dict(d, **{n: d[n] + s * step})).double()).sum()) for s in (1, -1)]
        slope = float((g[grad].double() * step.double()).sum())
        # each loss: N d_out outputs, each off by a few 2^-21 of terms of order 10
        assert abs((loss[0] - loss[1]) / 2 - slope) <= N * 40 * 10 * 2.0 ** -19, n


def test_adapter_tokens_do_not_reach_one_another():
    t = make(150, 264, 136, 4, 16, "bf16", "mixed", False, True)
    d = cuda(t)
    y, g = forward(d), backward(d)
    bad = 7
    a = int(t["ids"][bad]) if int(t["ids"][bad]) >= 0 else 0
    d["ids"][bad] = a
    y, g = forward(d), backward(d)
    d["x"][bad, 3] = float("nan")
    d["dy"][bad, 5] = float("inf")
    y2, g2 = forward(d), backward(d)
    rest = [i for i in range(150) if i != bad]
    assert torch.equal(y[rest], y2[rest]) and torch.equal(g["dx"][rest], g2["dx"][rest])
    others = [i for i in range(4) if i != a]
    assert torch.equal(g["dA"][others], g2["dA"][others]) and torch.equal(g["dB"][others], g2["dB"][others])
    assert bool(y2[bad].isnan().all())


@pytest.mark.parametrize("N", [3, 100])
def test_adapter_ids_out_of_range_count_as_none_and_are_reported(N):
    t = make(N, 64, 40, 2, 8, "bf16", "mixed", False, True)
    t["ids"][0], t["ids"][1] = 2, -7
    want, tol = reference(dict(t, ids=torch.where((t["ids"] < 0) | (t["ids"] > 1), -1, t["ids"])), True)
    d = cuda(t)
    ap = params(d)
    ws = workspace(moe.moe_adapter_workspace_size, ap, None)
    y = torch.empty(N, 40, device="cuda")
    moe.moe_adapter_forward(ap, d["x"], None, d["A"], d["B"], d["scale"], d["ids"], d["base"], y, ws)
    assert moe.moe_adapter_check(ap, ws) == moe.MOE_ERR_INVALID_ARG
    within("y", y, want["y"], tol["y"])
    d["ids"].clamp_(-1, 1)
    moe.moe_adapter_forward(ap, d["x"], None, d["A"], d["B"], d["scale"], d["ids"], d["base"], y, ws)
    assert moe.moe_adapter_check(ap, ws) == moe.MOE_OK


def test_adapter_empty_batch():
    ap = moe.adapter_params(0, 64, 40, 3, 8)
    ws = torch.full((moe.moe_adapter_backward_workspace_size(ap),), 0xFF, dtype=torch.uint8, device="cuda")
    L, p = moe.lib(), ctypes.byref(ap)
    dA, dB = torch.ones(3, 8, 64, device="cuda"), torch.ones(3, 40, 8, device="cuda")
    assert L.moe_adapter_forward(p, *[None] * 8, ws.data_ptr(), None) == moe.MOE_OK
    assert L.moe_adapter_backward(p, *[None] * 9, dA.data_ptr(), dB.data_ptr(), ws.data_ptr(), None) == moe.MOE_OK
    assert moe.moe_adapter_check(ap, ws) == moe.MOE_OK
    assert not dA.any() and not dB.any()


@pytest.mark.parametrize("N", [12, 140])
def test_adapters_in_a_graph_and_on_two_streams(N):
    first, second = (cuda(make(N, 264, 520, 6, 16, "bf16", "mixed", False, True, seed=s)) for s in (1, 2))
    want = [forward(first), forward(second)]
    grads = [backward(first), backward(second)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ys = []
    for _ in range(6):
        for s, d in ((s1, first), (s2, second)):
            with torch.cuda.stream(s):
                ap = params(d)
                ws = torch.empty(moe.moe_adapter_workspace_size(ap), dtype=torch.uint8, device="cuda")
                y = torch.empty(N, 520, device="cuda")
                moe.moe_adapter_forward(ap, d["x"], None, d["A"], d["B"], d["scale"], d["ids"], d["base"], y, ws)
                ys.append((y, ws))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 2]) for i, (y, _) in enumerate(ys))
    # captured, then replayed on another batch (another assignment of adapters too)
    d = {n: None if v is None else v.clone() for n, v in first.items()}
    ap = params(d)
    ws = torch.empty(moe.moe_adapter_workspace_size(ap), dtype=torch.uint8, device="cuda")
    bws = torch.empty(moe.moe_adapter_backward_workspace_size(ap), dtype=torch.uint8, device="cuda")
    y, dx = torch.empty(N, 520, device="cuda"), torch.empty(N, 264, device="cuda")
    dA, dB = torch.empty(d["A"].shape, device="cuda"), torch.empty(d["B"].shape, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_adapter_forward(ap, d["x"], None, d["A"], d["B"], d["scale"], d["ids"], d["base"], y, ws)
        moe.moe_adapter_backward(ap, d["x"], None, d["A"], d["B"], d["scale"], d["ids"], d["dy"], d["dx_base"], dx,
                                 dA, dB, bws)
    for i, batch in enumerate((first, second)):
        for n, v in batch.items():
            if v is not None:
                d[n].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i]) and torch.equal(dx, grads[i]["dx"])
        assert torch.equal(dA, grads[i]["dA"]) and torch.equal(dB, grads[i]["dB"])


@pytest.mark.parametrize("dtype,N", [("fp32", 20), ("fp32", 300), ("bf16", 300)])
def test_adapters_take_the_largest_finite_values(dtype, N):
    t = make(N, 136, 264, 3, 16, dtype, "mixed", False, False)
    bad = 11
    t["ids"][bad] = t["ids"][bad + 1] = 1
    top = torch.finfo(t["x"].dtype).max
    # values at the end of the range, through weights and beside factors that keep every result inside it
    t["x"][bad] *= 1e-3
    t["x"][bad + 1, 3], t["dy"][bad, 5] = top, torch.finfo(torch.float32).max
    t["A"][:, :, 3] *= 1e-3
    t["B"][:, 5] *= 1e-3
    t["dy"][bad + 1] *= 1e-3
    t["scale"][:] = 1e-3
    want, tol = reference(t, dtype == "bf16")
    assert all(bool((v.abs() < 3e38).all()) for v in want.values())
    d = cuda(t)
    got = dict(backward(d), y=forward(d))
    for n, v in want.items():
        within(n, got[n], v, tol[n])
