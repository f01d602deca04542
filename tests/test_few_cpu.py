"""Host-side checks of moe_forward_few (no call here reaches a CUDA device)."""
import ctypes

import pytest

import sparse_mixture_experts_25_b200 as moe

torch = pytest.importorskip("torch")

BASE = dict(N=8, d=64, d_f=96, E_r=4, k=2)


@pytest.mark.parametrize("kw,status", [
    (dict(N=33), moe.MOE_ERR_UNSUPPORTED),
    (dict(E_r=257), moe.MOE_ERR_UNSUPPORTED),
    (dict(c=1.0, reject_policy=moe.MOE_REJECT_REROUTE, reroute_depth=1), moe.MOE_ERR_UNSUPPORTED),
    (dict(c=1.0, accept_order=1), moe.MOE_ERR_UNSUPPORTED),
    (dict(E_r=256, d_f=65536), moe.MOE_ERR_UNSUPPORTED),
    (dict(E_r=255, d_f=65536, d_f_shared=65536), moe.MOE_ERR_UNSUPPORTED),
    (dict(d=1 << 24), moe.MOE_ERR_UNSUPPORTED),
    (dict(N=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(k=5), moe.MOE_ERR_INVALID_ARG),
])
def test_few_params_are_checked(kw, status):
    p = moe.params(**dict(BASE, **kw))
    with pytest.raises(moe.MoEError) as e:
        moe.moe_few_workspace_size(p)
    assert e.value.status == status
    call = moe.lib().moe_forward_few
    assert call(ctypes.byref(p), *[256] * 12, None) == status


def test_few_pointers_are_checked_before_any_device_work():
    L, q = moe.lib(), 256
    names = ("x", "W_r", "b_r", "lat", "W_g", "W_u", "W_d", "Ws_g", "Ws_u", "Ws_d", "Y", "ws")

    def call(p, **kw):
        return L.moe_forward_few(ctypes.byref(p), *[kw.get(n, q) for n in names], None)

    p = moe.params(**dict(BASE, d_f_shared=32))
    for n in ("x", "W_r", "W_g", "W_u", "W_d", "Ws_g", "Ws_u", "Ws_d", "Y"):
        assert call(p, **{n: None}) == call(p, **{n: q + 8}) == moe.MOE_ERR_INVALID_ARG, n
    assert call(p, ws=None) == call(p, ws=q + 8) == moe.MOE_ERR_WORKSPACE
    wlr = moe.params(**dict(BASE, norm=moe.MOE_NORM_WLR))
    assert call(wlr, lat=None) == moe.MOE_ERR_INVALID_ARG


def test_few_workspace_holds_the_forward_workspace_and_the_hidden_rows():
    p = moe.params(**BASE)
    assert moe.moe_few_workspace_size(p) >= moe.moe_workspace_size(p) + 8 * 2 * 96 * 6


def test_few_tensors_on_the_host_are_refused():
    p = moe.params(N=1, d=8, d_f=8, E_r=1, k=1, dtype=moe.MOE_F32)
    f = torch.zeros
    with pytest.raises(ValueError, match="host tensor"):
        moe.moe_forward_few(p, f(1, 8), f(1, 8), None, None, f(1, 8, 8), f(1, 8, 8), f(1, 8, 8), None, None, None,
                            f(1, 8), f(1 << 16, dtype=torch.uint8))
