"""Host logic of AdaptedLayer: on which device its calls are made.  No CUDA call
is made here: the library's functions are replaced by ones that note the device
that is current, and the tensors are host tensors, whose device stands for the
layer's."""
import contextlib

import pytest

import sparse_mixture_experts_25_b200 as moe

torch = pytest.importorskip("torch")

from sparse_mixture_experts_25_b200 import adapted  # noqa: E402

N, D, DF, E, ADAPTERS, RANK = 40, 64, 72, 4, 3, 8
CALLS = ("moe_forward", "moe_forward_few", "moe_adapter_forward", "moe_dropout_forward", "moe_dropout_backward",
         "moe_backward", "moe_adapter_backward", "moe_get_stats", "moe_adapter_check", "moe_backward_check")
RESULTS = {"moe_get_stats": (moe.MOE_OK, {}), "moe_adapter_check": moe.MOE_OK, "moe_backward_check": moe.MOE_OK}


@pytest.fixture
def made(monkeypatch):
    """Notes (call, current device) of every library call."""
    current, notes = ["another"], []

    @contextlib.contextmanager
    def device(d):
        current.append(d)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "device", device)
    for n in CALLS:
        monkeypatch.setattr(adapted, n, lambda *a, n=n, **k: (notes.append((n, current[-1])), RESULTS.get(n))[1])
    monkeypatch.setattr(adapted, "workspace_views", lambda p, ws: {"offsets": torch.zeros(E + 1, dtype=torch.int32)})
    monkeypatch.setattr(adapted, "moe_backward_workspace_size", lambda p, offsets: 256)
    return notes


def layer(n=N):
    f = torch.zeros
    p = moe.params(N=n, d=D, d_f=DF, E_r=E, k=2, dtype=moe.MOE_F32)
    w = {"W_r": f(E, D), "W_g": f(E, DF, D), "W_u": f(E, DF, D), "W_d": f(E, D, DF)}
    return adapted.AdaptedLayer(p, w, f(ADAPTERS, RANK, D), f(ADAPTERS, D, RANK), f(ADAPTERS))


def batch(n=N):
    return torch.zeros(n, D), torch.zeros(n, dtype=torch.int32), torch.zeros(n, D)


@pytest.mark.parametrize("n", [N, 7])
def test_every_call_is_made_on_the_layers_device(made, n):
    m = layer(n)
    m.forward(*batch(n))
    m.forward(*batch(n), training=True)
    m.backward(torch.zeros(n, D))
    m.check()
    names = {c for c, _ in made}
    assert names == set(CALLS) - ({"moe_forward_few"} if n > adapted.FEW_TOKENS else set())
    assert all(d == m.device for _, d in made), made


def test_tensors_of_another_device_are_refused(made):
    elsewhere = torch.zeros(N, D, device="meta")
    m = layer()
    x, ids, residual = batch()
    for bad in (dict(x=elsewhere), dict(residual=elsewhere), dict(ids=ids.to("meta")), dict(lat=elsewhere)):
        with pytest.raises(ValueError, match=next(iter(bad))):
            m.forward(**dict(dict(x=x, ids=ids, residual=residual), **bad))
    m.forward(x, ids, residual, training=True)
    with pytest.raises(ValueError, match="dout"):
        m.backward(elsewhere)
    made.clear()
    with pytest.raises(ValueError, match="scale"):
        adapted.AdaptedLayer(m.p, m.w, m.A, m.B, m.scale.to("meta"))
    with pytest.raises(ValueError, match="W_u"):
        adapted.AdaptedLayer(m.p, dict(m.w, W_u=m.w["W_u"].to("meta")), m.A, m.B, m.scale)
    assert not made


def test_check_reads_what_every_call_reported(made, monkeypatch):
    m = layer()
    with pytest.raises(ValueError, match="follows a forward"):  # nothing was written that it could read
        m.check()
    m.forward(*batch(), training=True)
    m.check()
    assert not any(n == "moe_backward_check" for n, _ in made)
    m.backward(torch.zeros(N, D))
    m.check()
    for bad, where in ((m.aws, "adapters"), (m.abws, "adapter gradients")):
        monkeypatch.setattr(adapted, "moe_adapter_check",
                            lambda ap, ws, bad=bad: moe.MOE_ERR_INVALID_ARG if ws is bad else moe.MOE_OK)
        with pytest.raises(moe.MoEError, match=where):
            m.check()
