"""The binding refuses a workspace that a call would write past (no call here
reaches a CUDA device: the tensors are stand-ins that only describe themselves)."""
import pytest

import sparse_mixture_experts_25_b200 as moe

torch = pytest.importorskip("torch")


class Described:
    """What the binding asks of a device tensor, without one."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, shape
        self.nbytes = torch.empty(0, dtype=dtype).element_size() * int(torch.Size(shape).numel())

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256


def adapter_tensors(ap, W):
    dt = torch.bfloat16 if ap.dtype == moe.MOE_BF16 else torch.float32
    f32 = torch.float32
    t = dict(x=Described(dt, ap.N, ap.d_in), W=Described(dt, ap.d_out, ap.d_in) if W else None,
             A=Described(dt, ap.n_adapters, ap.r, ap.d_in), B=Described(dt, ap.n_adapters, ap.d_out, ap.r),
             scale=Described(f32, ap.n_adapters), ids=Described(torch.int32, ap.N))
    forward = dict(t, base=None, y=Described(f32, ap.N, ap.d_out))
    backward = dict(t, dy=Described(f32, ap.N, ap.d_out), dx_base=None, dx=Described(f32, ap.N, ap.d_in),
                    dA=Described(f32, ap.n_adapters, ap.r, ap.d_in), dB=Described(f32, ap.n_adapters, ap.d_out, ap.r))
    return forward, backward


@pytest.mark.parametrize("N", [5, 700])
@pytest.mark.parametrize("W", [False, True])
def test_adapter_workspaces_are_measured(N, W):
    ap = moe.adapter_params(N, 64, 72, 4, 8)
    forward, backward = adapter_tensors(ap, W)
    for call, t, size in ((moe.moe_adapter_forward, forward, moe.moe_adapter_workspace_size),
                          (moe.moe_adapter_backward, backward, moe.moe_adapter_backward_workspace_size)):
        with pytest.raises(ValueError, match=f"workspace of {size(ap, W)} bytes"):
            call(ap, **t, ws=Described(torch.uint8, size(ap, W) - 1))
    if W:  # sized for the call without the projection
        with pytest.raises(ValueError, match="workspace of"):
            moe.moe_adapter_backward(ap, **backward, ws=Described(torch.uint8, moe.moe_adapter_backward_workspace_size(ap)))


def test_few_workspaces_are_measured():
    p = moe.params(N=8, d=64, d_f=96, E_r=4, k=2)
    bf, f32 = torch.bfloat16, torch.float32
    args = (Described(bf, 8, 64), Described(bf, 4, 64), None, None, Described(bf, 4, 96, 64), Described(bf, 4, 96, 64),
            Described(bf, 4, 64, 96), None, None, None, Described(f32, 8, 64))
    # the batch layer's workspace is smaller
    with pytest.raises(ValueError, match=f"workspace of {moe.moe_few_workspace_size(p)} bytes"):
        moe.moe_forward_few(p, *args, Described(torch.uint8, moe.moe_workspace_size(p)))
    # counted in bytes whatever the tensor's type is
    with pytest.raises(ValueError, match="workspace of"):
        moe.moe_forward_few(p, *args, Described(torch.int32, moe.moe_few_workspace_size(p) // 4 - 1))


@pytest.mark.parametrize("ws", [None, 256 + 8], ids=["missing", "misaligned address"])
def test_a_workspace_without_a_size_is_the_librarys_to_refuse(ws, monkeypatch):
    """None and plain addresses, which the binding takes too: the library's status."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    ap, p = moe.adapter_params(5, 64, 72, 4, 8), moe.params(N=8, d=64, d_f=96, E_r=4, k=2)
    forward, backward = adapter_tensors(ap, False)
    bf = torch.bfloat16
    few = (Described(bf, 8, 64), Described(bf, 4, 64), None, None, Described(bf, 4, 96, 64), Described(bf, 4, 96, 64),
           Described(bf, 4, 64, 96), None, None, None, Described(torch.float32, 8, 64))
    for call in (lambda: moe.moe_adapter_forward(ap, **forward, ws=ws, stream=0),
                 lambda: moe.moe_adapter_backward(ap, **backward, ws=ws, stream=0),
                 lambda: moe.moe_forward_few(p, *few, ws, stream=0)):
        with pytest.raises(moe.MoEError) as e:
            call()
        assert e.value.status == moe.MOE_ERR_WORKSPACE
