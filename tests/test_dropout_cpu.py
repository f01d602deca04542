"""Host-side checks of moe_dropout_* and the generator that the GPU tests use
(no call here reaches a CUDA device)."""
import ctypes

import numpy as np
import pytest

import sparse_mixture_experts_25_b200 as moe
from tests.philox import words

torch = pytest.importorskip("torch")


def test_generator_of_the_tests_gives_the_published_words():
    # known answers of Philox4x32-10 printed with the paper's code: counter and
    # key all zeros, all ones
    assert [hex(v) for v in words(np.array([0], np.uint64), 0, 0)[0]] == \
        ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    top = (1 << 64) - 1
    assert [hex(v) for v in words(np.array([top], np.uint64), top, top)[0]] == \
        ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(d=0), moe.MOE_ERR_INVALID_ARG),
    (dict(row0=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(rate=1.0), moe.MOE_ERR_INVALID_ARG),
    (dict(rate=-0.1), moe.MOE_ERR_INVALID_ARG),
    (dict(rate=float("nan")), moe.MOE_ERR_INVALID_ARG),
    (dict(dtype=2), moe.MOE_ERR_INVALID_ARG),
    (dict(d=36), moe.MOE_ERR_UNSUPPORTED),
    (dict(N=1 << 37), moe.MOE_ERR_UNSUPPORTED),
    (dict(row0=1 << 60), moe.MOE_ERR_UNSUPPORTED),
])
def test_dropout_params_are_checked(kw, status):
    assert ctypes.sizeof(moe.DropoutParams) == 48
    base = dict(N=4, d=64, rate=0.1)
    base.update(kw)
    dp, L = moe.dropout_params(**base), moe.lib()
    assert L.moe_dropout_forward(ctypes.byref(dp), 256, None, 256, None, None) == status
    assert L.moe_dropout_backward(ctypes.byref(dp), 256, 256, None, None) == status


def test_dropout_pointers_are_checked():
    dp, L = moe.dropout_params(4, 64, 0.1), moe.lib()
    p, bad = ctypes.byref(dp), moe.MOE_ERR_INVALID_ARG
    for Y, residual, out, step in ((None, None, 256, None), (256, None, None, None), (260, None, 256, None),
                                   (256, 264, 256, None), (256, None, 256, 260)):
        assert L.moe_dropout_forward(p, Y, residual, out, step, None) == bad
    for dout, dY, step in ((None, 256, None), (256, None, None), (256, 264, None), (256, 256, 4)):
        assert L.moe_dropout_backward(p, dout, dY, step, None) == bad
    assert L.moe_dropout_forward(ctypes.byref(moe.dropout_params(0, 64, 0.5)), None, None, None, None, None) == moe.MOE_OK


def test_dropout_tensors_are_checked_by_the_binding():
    dp = moe.dropout_params(2, 8, 0.5)
    f, h = torch.zeros(2, 8), torch.zeros(2, 8, dtype=torch.bfloat16)
    for Y, residual, out in ((h, None, h), (f, f, h), (f, None, f), (f, None, h[:1])):
        with pytest.raises(ValueError):
            moe.moe_dropout_forward(dp, Y, residual, out)
    with pytest.raises(ValueError, match="step"):
        moe.moe_dropout_backward(dp, h, f, step=torch.zeros(1))
    with pytest.raises(ValueError, match="host tensor"):
        moe.moe_dropout_forward(dp, f, None, h)
