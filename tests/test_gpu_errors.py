"""A call that the CUDA runtime refuses reports it by its status; the program's
next call must not be given the same error again.  The refusal here: a call that
waits for its stream, on a stream that is being captured."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - GPU tests need a device
    pytest.skip("no CUDA device", allow_module_level=True)

import sparse_mixture_experts_25_b200 as moe  # noqa: E402


@pytest.mark.parametrize("name", ["moe_get_stats", "moe_adapter_check"])
def test_a_refused_call_leaves_no_error_behind(name):
    p, ap = moe.params(N=8, d=64, d_f=96, E_r=4, k=2), moe.adapter_params(16, 64, 72, 4, 8)
    size = moe.moe_workspace_size(p) if name == "moe_get_stats" else moe.moe_adapter_workspace_size(ap)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    runtime = ctypes.CDLL("libcudart.so.12")  # the one that the library is linked with
    raw, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    assert runtime.cudaStreamBeginCapture(raw, 1) == 0
    try:
        if name == "moe_get_stats":
            status = moe.lib().moe_get_stats(ctypes.byref(p), ws.data_ptr(), ctypes.byref(moe.Stats()),
                                             stream.cuda_stream)
        else:
            status = moe.moe_adapter_check(ap, ws, stream)
        left = runtime.cudaPeekAtLastError()
    finally:
        runtime.cudaStreamEndCapture(raw, ctypes.byref(graph))
        runtime.cudaGetLastError()
    assert status == moe.MOE_ERR_CUDA and moe.lib().moe_last_error().decode().startswith(name)
    assert left == 0
    assert float(torch.ones(4, device="cuda").sum()) == 4
