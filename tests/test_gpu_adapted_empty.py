"""A step of AdaptedLayer without tokens: nothing to write but the weights'
gradients, which are zero, and nothing to report, whatever the workspaces held."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - GPU tests need a device
    pytest.skip("no CUDA device", allow_module_level=True)

import sparse_mixture_experts_25_b200 as moe  # noqa: E402
from sparse_mixture_experts_25_b200.adapted import AdaptedLayer  # noqa: E402


@pytest.mark.parametrize("shared", [0, 40])
@pytest.mark.parametrize("dtype", [moe.MOE_BF16, moe.MOE_F32])
def test_steps_of_an_empty_batch(dtype, shared, monkeypatch):
    dt = torch.bfloat16 if dtype == moe.MOE_BF16 else torch.float32
    d, d_f, E, a, r = 64, 72, 4, 3, 8

    def rand(*shape):
        return torch.randn(shape, device="cuda").to(dt)

    w = {"W_r": rand(E, d), "b_r": torch.zeros(E, device="cuda"), "W_g": rand(E, d_f, d), "W_u": rand(E, d_f, d),
         "W_d": rand(E, d, d_f)}
    if shared:
        w.update(Ws_g=rand(shared, d), Ws_u=rand(shared, d), Ws_d=rand(d, shared))
    p = moe.params(N=0, d=d, d_f=d_f, E_r=E, k=2, dtype=dtype, d_f_shared=shared)
    empty = torch.empty

    def filled(*size, **kw):  # what a workspace or an output may hold before the call
        t = empty(*size, **kw)
        t.view(torch.uint8).fill_(0xFF) if t.dim() and t.numel() else None
        return t

    monkeypatch.setattr(torch, "empty", filled)
    layer = AdaptedLayer(p, w, rand(a, r, d), rand(a, d, r), torch.ones(a, device="cuda"), rate=0.5, seed=3)
    x, ids, residual = rand(0, d), torch.zeros(0, dtype=torch.int32, device="cuda"), rand(0, d)
    for training in (False, True):
        assert layer.forward(x, ids, residual, training=training).shape == (0, d)
        assert layer.check()["requested"] == 0
    g = layer.backward(rand(0, d))
    assert layer.check()["requested"] == 0
    assert set(g) == {"dx", "dA", "dB"} | {"d" + n for n in w}
    assert all(not t.any() for t in g.values())
