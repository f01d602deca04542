"""Host-side checks of moe_adapter_* (no call here reaches a CUDA device)."""
import ctypes

import pytest

import sparse_mixture_experts_25_b200 as moe

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(d_in=0), moe.MOE_ERR_INVALID_ARG),
    (dict(n_adapters=0), moe.MOE_ERR_INVALID_ARG),
    (dict(r=0), moe.MOE_ERR_INVALID_ARG),
    (dict(dtype=4), moe.MOE_ERR_INVALID_ARG),
    (dict(d_in=60), moe.MOE_ERR_UNSUPPORTED),
    (dict(d_out=65), moe.MOE_ERR_UNSUPPORTED),
    (dict(r=12), moe.MOE_ERR_UNSUPPORTED),
    (dict(r=136), moe.MOE_ERR_UNSUPPORTED),
    (dict(n_adapters=1025), moe.MOE_ERR_UNSUPPORTED),
    (dict(N=1 << 30), moe.MOE_ERR_UNSUPPORTED),
])
def test_adapter_params_are_checked(kw, status):
    base = dict(N=16, d_in=64, d_out=72, n_adapters=4, r=8)
    base.update(kw)
    ap = moe.adapter_params(**base)
    for size in (moe.moe_adapter_workspace_size, moe.moe_adapter_backward_workspace_size):
        with pytest.raises(moe.MoEError) as e:
            size(ap)
        assert e.value.status == status


def test_adapter_pointers_are_checked_before_any_device_work():
    assert ctypes.sizeof(moe.AdapterParams) == 32
    ap = moe.adapter_params(16, 64, 72, 4, 8)
    L, p, q = moe.lib(), ctypes.byref(ap), 256

    def forward(x=q, W=None, A=q, B=q, scale=q, ids=q, base=None, y=q, ws=q):
        return L.moe_adapter_forward(p, x, W, A, B, scale, ids, base, y, ws, None)

    def backward(x=q, W=None, A=q, B=q, scale=q, ids=q, dy=q, dx_base=None, dx=q, dA=q, dB=q, ws=q):
        return L.moe_adapter_backward(p, x, W, A, B, scale, ids, dy, dx_base, dx, dA, dB, ws, None)

    for call, names in ((forward, ("x", "A", "B", "scale", "ids", "y")),
                        (backward, ("x", "A", "B", "scale", "ids", "dy", "dx", "dA", "dB"))):
        for n in names:
            assert call(**{n: None}) == moe.MOE_ERR_INVALID_ARG, n
        for n in set(names) - {"scale", "ids"}:
            assert call(**{n: q + 4}) == moe.MOE_ERR_INVALID_ARG, n
        assert call(ws=None) == call(ws=q + 8) == moe.MOE_ERR_WORKSPACE
    # the projection is written to y before base is added
    assert forward(W=q, base=512, y=512) == moe.MOE_ERR_INVALID_ARG
    assert backward(W=q, dx_base=512, dx=512) == moe.MOE_ERR_INVALID_ARG
    big = moe.adapter_params(65535 * 64 + 1, 64, 72, 4, 8, dtype=moe.MOE_F32)
    assert L.moe_adapter_forward(ctypes.byref(big), q, q, q, q, q, q, None, q, q, None) == moe.MOE_ERR_UNSUPPORTED


def test_adapter_workspace_grows_with_what_the_call_needs():
    ap = moe.adapter_params(1000, 4096, 2048, 4, 16)
    f, b = moe.moe_adapter_workspace_size(ap), moe.moe_adapter_backward_workspace_size(ap)
    assert f >= 1000 * (4 + 2 * 2 * 16) and b >= f + 1000 * 2 * 2 * 16
    assert moe.moe_adapter_backward_workspace_size(ap, True) >= b + 2 * 2 * 1000 * 2048
    assert moe.moe_adapter_workspace_size(ap, True) == f


def test_adapter_tensors_are_checked_by_the_binding():
    ap = moe.adapter_params(4, 16, 24, 2, 8, dtype=moe.MOE_F32)
    t = dict(x=torch.zeros(4, 16), W=None, A=torch.zeros(2, 8, 16), B=torch.zeros(2, 24, 8), scale=torch.zeros(2),
             ids=torch.zeros(4, dtype=torch.int32), base=None, y=torch.zeros(4, 24), ws=torch.zeros(1 << 16, dtype=torch.uint8))
    for name, bad in (("x", torch.zeros(4, 24)), ("A", torch.zeros(2, 16, 8)), ("B", torch.zeros(2, 8, 24)),
                      ("ids", torch.zeros(4, dtype=torch.int64)), ("scale", torch.zeros(2, dtype=torch.float64)),
                      ("x", torch.zeros(4, 16, dtype=torch.bfloat16)), ("y", torch.zeros(4, 16)),
                      ("W", torch.zeros(16, 24))):
        with pytest.raises(ValueError, match=name):
            moe.moe_adapter_forward(ap, **dict(t, **{name: bad}))
    with pytest.raises(ValueError, match="host tensor"):
        moe.moe_adapter_forward(ap, **t)
