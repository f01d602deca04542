"""Cases for the operators that fine-tune and serve the sparse MoE layer.

Three operators that are used next to one another:

  few      the whole layer for a batch of a few tokens (moe_forward_few)
  adapter  low-rank adapters of many requests beside a shared projection or
           beside the layer (moe_adapter_forward, moe_adapter_backward)
  dropout  dropout of the layer's output in front of the residual sum, its mask
           a function of a counter and never stored (moe_dropout_forward,
           moe_dropout_backward)

`run` computes them in elementary torch operations while `own` is false, and
through the package's entry points while it is true.
"""
import math

import torch

own = False

RENORM, FULLPROB = 0, 1
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _few(N, d, d_f, E, k, d_sh=0, c=0.0, norm=RENORM, bias=False, dtype="bf16"):
    return {"op": "few", "N": N, "d": d, "d_f": d_f, "E": E, "k": k, "d_sh": d_sh, "c": c, "norm": norm,
            "bias": bias, "dtype": dtype}


def _adapter(N, d_in, d_out, n_adapters, r, W=False, base=True, runs=True, backward=False, dtype="bf16"):
    return {"op": "adapter", "N": N, "d_in": d_in, "d_out": d_out, "n_adapters": n_adapters, "r": r, "W": W,
            "base": base, "runs": runs, "backward": backward, "dtype": dtype}


def _dropout(N, d, rate, residual=True, backward=False, row0=0, dtype="bf16"):
    return {"op": "dropout", "N": N, "d": d, "rate": rate, "residual": residual, "backward": backward,
            "row0": row0, "dtype": dtype}


def listed():
    return [
        # one token through a small fp32 top-1 layer with full-probability weights:
        # nothing but latency
        dict(_few(1, 256, 512, 8, 1, norm=FULLPROB, dtype="fp32"), name="few: 1 token fp32 top-1"),
        # one token of one sequence through a layer of 128 narrow experts with a router bias
        dict(_few(1, 4096, 1536, 128, 8, bias=True), name="few: 1 token 128 experts"),
        # a small batch of sequences over eight wide experts: all of them are read
        dict(_few(7, 4096, 14336, 8, 2), name="few: 7 tokens wide experts"),
        # the largest batch: most of 256 experts, an always-on shared expert, and a capacity limit
        dict(_few(32, 7168, 2048, 256, 8, d_sh=2048, c=2.0), name="few: 32 tokens 256 experts"),
        # one new token of each of 16 requests, each with an adapter of its own, beside
        # the layer: the adapters' output is added to the layer's
        dict(_adapter(16, 4096, 4096, 64, 16, runs=False), name="adapter: 16 requests"),
        # prompts of up to 32 adapters through a shared projection
        dict(_adapter(4096, 4096, 4096, 32, 16, W=True, base=False), name="adapter: prompts projection"),
        # fp32, a ragged batch whose tokens are in no order, ranks of 40
        dict(_adapter(1531, 1000, 2056, 7, 40, runs=False, dtype="fp32"), name="adapter: fp32 mixed tokens"),
        # gradients of four adapters beside the layer, long prompts, ranks of 64
        dict(_adapter(8192, 4096, 4096, 4, 64, backward=True), name="adapter grads: beside the layer"),
        # gradients of 16 adapters and of x through a shared projection
        dict(_adapter(2047, 4096, 1536, 16, 16, W=True, base=False, backward=True),
             name="adapter grads: projection"),
        # one decoding-sized batch in fp32: latency
        dict(_dropout(17, 1024, 0.1, dtype="fp32"), name="dropout: 17 rows fp32"),
        # a training batch, bf16 residual stream
        dict(_dropout(8192, 4096, 0.1), name="dropout: 8192 rows"),
        # the same batch's gradient, as a later shard of the routing group
        dict(_dropout(8191, 7168, 0.25, backward=True, row0=8192), name="dropout grads: 8191 rows"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["few", "few", "adapter", "adapter", "dropout"])
    if op == "few":
        for _ in range(1000):
            E = _log(rng, 2, 256)
            case = _few(_log(rng, 1, 32), _log(rng, 64, 7168, 8), _log(rng, 64, 14336, 8), E,
                        rng.randint(1, min(E, 8)), d_sh=rng.choice([0, 0, _log(rng, 64, 4096, 8)]),
                        c=rng.choice([0.0, 0.0, 1.0, 1.5]), norm=rng.choice([RENORM, RENORM, FULLPROB]),
                        bias=rng.random() < 0.3, dtype=rng.choice(["bf16", "bf16", "bf16", "fp32"]))
            size = (2 if case["dtype"] == "bf16" else 4) * 3 * case["d"] * (case["d_f"] * E + case["d_sh"])
            if size <= 12e9:
                return case
        return case
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "adapter":
        backward = rng.random() < 0.5
        W = dtype == "bf16" and rng.random() < 0.4
        r = rng.choice([8, 8, 16, 16, 24, 32, 40, 64])
        most = 4096 if dtype == "bf16" else 2048
        N = _log(rng, 1, most)
        return _adapter(N, _log(rng, 64, 4096, 8), _log(rng, 64, 4096, 8), _log(rng, 1, 64), r, W=W,
                        base=rng.random() < 0.5, runs=rng.random() < 0.5, backward=backward, dtype=dtype)
    return _dropout(_log(rng, 1, 8192), _log(rng, 64, 7168, 8), rng.choice([0.05, 0.1, 0.25, 0.5]),
                    residual=rng.random() < 0.8, backward=rng.random() < 0.5,
                    row0=rng.choice([0, rng.randint(1, 1 << 20)]), dtype=dtype)


def _elements(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    s = _elements(case)
    if case["op"] == "few":
        N, d, d_f, E, k = (case[n] for n in ("N", "d", "d_f", "E", "k"))
        touched = E * (1 - (1 - k / E) ** N)          # experts that some token chose, on average
        size = s * (3 * touched * d_f * d + E * d + 3 * case["d_sh"] * d + N * d) + 4 * N * d + 8 * N * k
        return {"bytes": size, "flops": 2 * N * (3 * k * d_f * d + E * d + 3 * case["d_sh"] * d)}
    if case["op"] == "adapter":
        N, i, o, a, r = (case[n] for n in ("N", "d_in", "d_out", "n_adapters", "r"))
        used = a * (1 - (1 - 1 / (a + 1)) ** N)       # adapters that some token has, on average
        size = s * (N * i + used * r * (i + o)) + 4 * N
        flops = 2 * N * r * (i + o)
        if not case["backward"]:
            size += 4 * N * o * (2 if case["base"] else 1)
        else:
            size += 4 * (N * o + N * i * (2 if case["base"] else 1) + a * r * (i + o))
            flops *= 3
        if case["W"]:
            size += s * i * o
            flops += 2 * N * i * o
        return {"bytes": size, "flops": flops}
    n = case["N"] * case["d"]
    if case["backward"]:
        return {"bytes": n * (s + 4), "flops": n}
    return {"bytes": n * (4 + s * (2 if case["residual"] else 1)), "flops": 2 * n}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _normal(g, std, dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _routable(g, N, d, k, W_r, b_r, dtype):
    """Token rows whose first k + 1 scores are apart: the ranks do not hang on the order of a sum."""
    x = _normal(g, 1.0, dtype, N, d)
    k1 = min(k + 1, W_r.shape[0])
    for _ in range(50):
        scores = x.double() @ W_r.double().T + (0 if b_r is None else b_r.double())
        top = scores.topk(k1, dim=1).values
        near = (top[:, :-1] - top[:, 1:] < 1e-4).any(dim=1) if k1 > 1 else torch.zeros(N, dtype=torch.bool)
        if not bool(near.any()):
            break
        x = torch.where(near[:, None], _normal(g, 1.0, dtype, N, d), x)
    return x


def _few_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    N, d, d_f, E, k, d_sh = (case[n] for n in ("N", "d", "d_f", "E", "k", "d_sh"))
    t = {"W_r": _normal(g, d ** -0.5, dt, E, d), "b_r": None, "Ws_g": None, "Ws_u": None, "Ws_d": None}
    if case["bias"]:  # hot experts: half the logarithm of a Zipf share
        share = torch.arange(1, E + 1, device="cuda", dtype=torch.float32) ** -1.2
        t["b_r"] = (0.5 * (share / share.sum()).log())[torch.randperm(E, generator=g, device="cuda")].contiguous()
    t["x"] = _routable(g, N, d, k, t["W_r"], t["b_r"], dt)
    t["W_g"] = _normal(g, d ** -0.5, dt, E, d_f, d)
    t["W_u"] = _normal(g, d ** -0.5, dt, E, d_f, d)
    t["W_d"] = _normal(g, d_f ** -0.5, dt, E, d, d_f)
    if d_sh:
        t["Ws_g"] = _normal(g, d ** -0.5, dt, d_sh, d)
        t["Ws_u"] = _normal(g, d ** -0.5, dt, d_sh, d)
        t["Ws_d"] = _normal(g, d_sh ** -0.5, dt, d, d_sh)
    return t


def _adapter_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    N, i, o, a, r = (case[n] for n in ("N", "d_in", "d_out", "n_adapters", "r"))
    # one adapter in a + 1 draws is none (-1); `runs`: a request's tokens follow one another
    ids = torch.randint(-1, a, (N,), generator=g, device="cuda", dtype=torch.int32)
    if case["runs"]:
        cut = torch.rand(N, generator=g, device="cuda") < min(1.0, 2 * a / N)
        start = torch.cummax(torch.where(cut, torch.arange(N, device="cuda"), 0), 0).values
        ids = ids[start].contiguous()
    t = {"ids": ids, "scale": torch.rand(a, generator=g, device="cuda") + 0.5,
         "A": _normal(g, i ** -0.5, dt, a, r, i), "B": _normal(g, r ** -0.5, dt, a, o, r),
         "x": _normal(g, 1.0, dt, N, i), "W": _normal(g, i ** -0.5, dt, o, i) if case["W"] else None,
         "base": None}
    if case["backward"]:
        t["dy"] = _normal(g, 1.0, torch.float32, N, o)
        t["base"] = _normal(g, 1.0, torch.float32, N, i) if case["base"] else None
    else:
        t["base"] = _normal(g, 1.0, torch.float32, N, o) if case["base"] else None
    return t


def _dropout_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    N, d = case["N"], case["d"]
    t = {"seed": 0x9E3779B97F4A7C15 ^ (seed * 0x100000001), "offset": (seed << 3) + 5}
    if case["backward"]:
        t["dout"] = _normal(g, 1.0, dt, N, d)
    else:
        t["Y"] = _normal(g, 1.0, torch.float32, N, d)
        t["residual"] = _normal(g, 2.0, dt, N, d) if case["residual"] else None
    return t


def prepare(case, seed):
    make = {"few": _few_inputs, "adapter": _adapter_inputs, "dropout": _dropout_inputs}[case["op"]]
    s = {"case": case, **make(case, seed)}
    if own:
        # what a program keeps over its calls: the parameters, the workspace, the outputs
        import sparse_mixture_experts_25_b200 as moe

        dt = moe.MOE_BF16 if case["dtype"] == "bf16" else moe.MOE_F32
        if case["op"] == "few":
            p = moe.params(case["N"], case["d"], case["d_f"], case["E"], case["k"], c=case["c"],
                           norm=case["norm"], dtype=dt, d_f_shared=case["d_sh"])
            ws = torch.empty(moe.moe_few_workspace_size(p), dtype=torch.uint8, device="cuda")
            views = moe.workspace_views(p, ws)
            s.update(p=p, ws=ws, Y=torch.empty(case["N"], case["d"], device="cuda"), rec_ids=views["ids"],
                     rec_w=views["w"])
        elif case["op"] == "adapter":
            p = moe.adapter_params(case["N"], case["d_in"], case["d_out"], case["n_adapters"], case["r"], dtype=dt)
            size = moe.moe_adapter_backward_workspace_size if case["backward"] else moe.moe_adapter_workspace_size
            s.update(p=p, ws=torch.empty(size(p, case["W"]), dtype=torch.uint8, device="cuda"))
            if case["backward"]:
                s.update(dx=torch.empty(case["N"], case["d_in"], device="cuda"),
                         dA=torch.empty(s["A"].shape, device="cuda"), dB=torch.empty(s["B"].shape, device="cuda"))
            else:
                s.update(y=torch.empty(case["N"], case["d_out"], device="cuda"))
        else:
            s["p"] = moe.dropout_params(case["N"], case["d"], case["rate"], seed=s["seed"], offset=s["offset"],
                                        row0=case["row0"], dtype=dt)
            out = torch.float32 if case["backward"] else DTYPES[case["dtype"]]
            s["out"] = torch.empty(case["N"], case["d"], dtype=out, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _silu(z):
    return z / (1 + torch.exp(-z))


def _capacity(case):
    N, k, E, c = case["N"], case["k"], case["E"], case["c"]
    return N if c <= 0 else max(1, math.ceil(c * N * k / E - 1e-9))


def _plain_few(s):
    case = s["case"]
    N, E, k = case["N"], case["E"], case["k"]
    x = s["x"].float()
    scores = s["x"].double() @ s["W_r"].double().T
    if s["b_r"] is not None:
        scores = scores + s["b_r"].double()
    e = torch.exp(scores - scores.max(dim=1, keepdim=True).values)
    ids = torch.sort(scores, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = torch.gather(e, 1, ids)
    w = chosen / (chosen if case["norm"] == RENORM else e).sum(dim=1, keepdim=True)
    # an expert takes its first C requests in token order
    asked = torch.zeros(N, E, dtype=torch.int64, device="cuda").scatter_(1, ids, 1)
    taken = torch.gather(torch.cumsum(asked, 0), 1, ids) <= _capacity(case)
    cw = torch.where(taken, w, torch.zeros_like(w)).float()
    if N * k < E:  # the chosen experts' weights, path by path
        at = ids.reshape(-1)
        xr = x.repeat_interleave(k, 0)[:, :, None]
        h = _silu(torch.bmm(s["W_g"][at].float(), xr)) * torch.bmm(s["W_u"][at].float(), xr)
        paths = torch.bmm(s["W_d"][at].float(), h)[:, :, 0].reshape(N, k, -1)
        Y = (cw[:, :, None] * paths).sum(dim=1)
    else:          # every expert on every token, masked by the weights
        h = _silu(torch.matmul(x, s["W_g"].float().transpose(1, 2)))
        h = h * torch.matmul(x, s["W_u"].float().transpose(1, 2))
        outs = torch.matmul(h, s["W_d"].float().transpose(1, 2))
        dense = torch.zeros(N, E, device="cuda").scatter_(1, ids, cw)
        Y = torch.einsum("ne,end->nd", dense, outs)
    if s["Ws_g"] is not None:
        h = _silu(x @ s["Ws_g"].float().T) * (x @ s["Ws_u"].float().T)
        Y = Y + h @ s["Ws_d"].float().T
    return {"Y": Y, "ids": ids.int(), "w": w.float()}


def _plain_adapter(s):
    # all adapters side by side as one low-rank pair; a token's row is masked to its own adapter
    case = s["case"]
    N, a, r = case["N"], case["n_adapters"], case["r"]
    x, A, B = s["x"].float(), s["A"].float().reshape(a * r, -1), s["B"].float()
    Bt = B.transpose(1, 2).reshape(a * r, -1)
    mask = (s["ids"][:, None] == torch.arange(a, device="cuda")[None, :]).float() * s["scale"][None, :]
    mask = mask[:, :, None].expand(N, a, r).reshape(N, a * r)
    U = (x @ A.T) * mask
    if not case["backward"]:
        y = U @ Bt
        if s["W"] is not None:
            y = y + x @ s["W"].float().T
        return {"y": y if s["base"] is None else y + s["base"]}
    V = (s["dy"] @ Bt.T) * mask
    dx = V @ A
    if s["W"] is not None:
        dx = dx + s["dy"] @ s["W"].float()
    return {"dx": dx if s["base"] is None else dx + s["base"], "dA": (V.T @ x).reshape(s["A"].shape),
            "dB": (U.T @ s["dy"]).reshape(a, r, -1).transpose(1, 2).contiguous()}


M32 = 0xFFFFFFFF


def _philox(group, key, offset):
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011): four words for each 64-bit counter."""
    c0, c1 = group & M32, group >> 32
    c2, c3 = torch.full_like(group, offset & M32), torch.full_like(group, offset >> 32 & M32)
    k0, k1 = key & M32, key >> 32 & M32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57      # the low 64 bits are those of the unsigned product
        c0, c1, c2, c3 = (p1 >> 32 & M32) ^ c1 ^ k0, p1 & M32, (p0 >> 32 & M32) ^ c3 ^ k1, p0 & M32
        k0, k1 = k0 + 0x9E3779B9 & M32, k1 + 0xBB67AE85 & M32
    return torch.stack([c0, c1, c2, c3], dim=1)


def _kept(case, s):
    n = case["N"] * case["d"]
    first = case["row0"] * case["d"] // 4
    words = _philox(torch.arange(first, first + n // 4, device="cuda"), s["seed"], s["offset"])
    return (words >= round(case["rate"] * 2 ** 32)).reshape(case["N"], case["d"])


def _plain_dropout(s):
    case = s["case"]
    kept = _kept(case, s)
    scale = 1.0 / (1.0 - case["rate"])
    if case["backward"]:
        dout = s["dout"].float()
        return {"dY": torch.where(kept, dout * scale, torch.zeros_like(dout))}
    out = torch.where(kept, s["Y"] * scale, torch.zeros_like(s["Y"]))
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return {"out": out.to(DTYPES[case["dtype"]])}


def _own(s):
    import sparse_mixture_experts_25_b200 as moe

    case = s["case"]
    if case["op"] == "few":
        moe.moe_forward_few(s["p"], s["x"], s["W_r"], s["b_r"], None, s["W_g"], s["W_u"], s["W_d"], s["Ws_g"],
                            s["Ws_u"], s["Ws_d"], s["Y"], s["ws"])
        return {"Y": s["Y"], "ids": s["rec_ids"], "w": s["rec_w"]}
    if case["op"] == "adapter":
        if case["backward"]:
            moe.moe_adapter_backward(s["p"], s["x"], s["W"], s["A"], s["B"], s["scale"], s["ids"], s["dy"],
                                     s["base"], s["dx"], s["dA"], s["dB"], s["ws"])
            return {"dx": s["dx"], "dA": s["dA"], "dB": s["dB"]}
        moe.moe_adapter_forward(s["p"], s["x"], s["W"], s["A"], s["B"], s["scale"], s["ids"], s["base"], s["y"],
                                s["ws"])
        return {"y": s["y"]}
    if case["backward"]:
        moe.moe_dropout_backward(s["p"], s["dout"], s["out"])
        return {"dY": s["out"]}
    moe.moe_dropout_forward(s["p"], s["Y"], s["residual"], s["out"])
    return {"out": s["out"]}


def run(state):
    if own:
        return _own(state)
    return {"few": _plain_few, "adapter": _plain_adapter, "dropout": _plain_dropout}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "few":
        return _exact_few(case, _few_inputs(case, seed))
    if case["op"] == "adapter":
        return _exact_adapter(case, _adapter_inputs(case, seed))
    return _exact_dropout(case, _dropout_inputs(case, seed))


def _exact_few(case, t):
    """Algorithm by algorithm, token by token: scores, the k largest, slots in token order, expert by expert."""
    N, E, k = case["N"], case["E"], case["k"]
    x = t["x"].double()
    g = torch.stack([x @ t["W_r"][e].double() for e in range(E)], dim=1)
    if t["b_r"] is not None:
        g += t["b_r"].double()
    g = g.cpu()
    p = torch.softmax(g, dim=1)
    ids = torch.empty(N, k, dtype=torch.int32)
    w = torch.empty(N, k, dtype=torch.float64)
    rows = {}
    for n in range(N):
        order = sorted(range(E), key=lambda e: (-float(g[n, e]), e))[:k]
        total = sum(float(p[n, e]) for e in order) if case["norm"] == RENORM else 1.0
        for j, e in enumerate(order):
            ids[n, j], w[n, j] = e, float(p[n, e]) / total
            rows.setdefault(e, []).append((n, float(p[n, e]) / total))
    Y = torch.zeros_like(x)
    for e, paths in rows.items():
        paths = paths[:_capacity(case)]
        at = torch.tensor([n for n, _ in paths], device="cuda")
        a = torch.tensor([v for _, v in paths], device="cuda", dtype=torch.float64)
        z = x[at] @ t["W_g"][e].double().T
        h = z * torch.sigmoid(z) * (x[at] @ t["W_u"][e].double().T)
        Y.index_add_(0, at, a[:, None] * (h @ t["W_d"][e].double().T))
    if t["Ws_g"] is not None:
        z = x @ t["Ws_g"].double().T
        Y += (z * torch.sigmoid(z) * (x @ t["Ws_u"].double().T)) @ t["Ws_d"].double().T
    return {"Y": Y, "ids": ids, "w": w}


def _exact_adapter(case, t):
    """Adapter by adapter, on the rows that have it."""
    ids = t["ids"].cpu()
    x = t["x"].double()
    W = None if t["W"] is None else t["W"].double()
    if not case["backward"]:
        y = torch.zeros(case["N"], case["d_out"], dtype=torch.float64, device="cuda")
    else:
        dy = t["dy"].double()
        y = torch.zeros_like(x)
        dA, dB = torch.zeros_like(t["A"], dtype=torch.float64), torch.zeros_like(t["B"], dtype=torch.float64)
    if t["base"] is not None:
        y += t["base"].double()
    if W is not None:
        y += dy @ W if case["backward"] else x @ W.T
    for a in range(case["n_adapters"]):
        at = torch.nonzero(ids == a).reshape(-1).cuda()
        if not len(at):
            continue
        A, B, s = t["A"][a].double(), t["B"][a].double(), float(t["scale"][a])
        if not case["backward"]:
            y[at] += s * ((x[at] @ A.T) @ B.T)
        else:
            y[at] += s * ((dy[at] @ B) @ A)
            dA[a] = s * ((dy[at] @ B).T @ x[at])
            dB[a] = s * (dy[at].T @ (x[at] @ A.T))
    return {"dx": y, "dA": dA, "dB": dB} if case["backward"] else {"y": y}


def _exact_dropout(case, t):
    """The same generator in numpy's unsigned arithmetic, then the sum in 64 bits."""
    import numpy as np

    n = case["N"] * case["d"]
    i = np.arange(n // 4, dtype=np.uint64) + np.uint64(case["row0"] * case["d"] // 4)
    low, half = np.uint64(M32), np.uint64(32)
    c = [i & low, i >> half, np.uint64(t["offset"] & M32), np.uint64(t["offset"] >> 32 & M32)]
    key = [t["seed"] & M32, t["seed"] >> 32 & M32]
    for r in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ np.uint64((key[0] + r * 0x9E3779B9) & M32), b & low,
             (a >> half) ^ c[3] ^ np.uint64((key[1] + r * 0xBB67AE85) & M32), a & low]
    kept = torch.empty(n // 4, 4, dtype=torch.bool)
    for j in range(4):
        kept[:, j] = torch.from_numpy(np.broadcast_to(c[j], i.shape) >= np.uint64(round(case["rate"] * 2 ** 32)))
    kept = kept.reshape(case["N"], case["d"]).cuda().double()
    if case["backward"]:
        return {"dY": kept * t["dout"].double() / (1 - case["rate"])}
    out = kept * t["Y"].double() / (1 - case["rate"])
    return {"out": out if t["residual"] is None else out + t["residual"].double()}
