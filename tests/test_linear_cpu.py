"""The dense 4-bit linear without a GPU: its oracle on worked weights, and every
refusal, made before the first CUDA call."""
import numpy as np
import pytest
import torch

from oracle import linear as O


@pytest.fixture(scope="module")
def moe():
    from expert_offload_serving_b200 import build
    build.build()
    import expert_offload_serving_b200 as m
    m.lib()
    return m


def test_int4_weights_by_hand():
    codes = np.array([[0x10, 0xF8]], dtype=np.uint8)                  # codes 0, 1, 8, 15
    w = O.dequant_int4(np.repeat(codes, 16, axis=1), [[0.5, 2.0]], 32, [[8, 3]])
    assert w.shape == (1, 64)
    assert w[0, 0] == -4.0 and w[0, 1] == -3.5                         # 0.5 * (0 - 8), 0.5 * (1 - 8)
    assert w[0, 32] == 10.0 and w[0, 33] == 24.0                       # 2 * (8 - 3), 2 * (15 - 3)
    assert np.array_equal(O.dequant_int4(codes, [[1.0]], 32), [[-8.0, -7.0, 0.0, 7.0]])


def test_swiglu_and_accumulate_by_hand():
    w = np.array([[1.0, 0.0], [0.0, 1.0]])
    y = O.linear([[2.0, 3.0]], w, swiglu=True, y0=[[1.0]])
    assert abs(y[0, 0] - (1.0 + 2.0 / (1 + np.exp(-2.0)) * 3.0)) < 1e-15


def _call(moe, p, N=16, K=64, fmt=3, group=32, st=1, codes=0, scales=0, zeros=None, x=0, xt=1, ldx=64, T=2, y=0, yt=0,
          ldy=16, flags=0):
    at = lambda v: None if v is None else p + v
    return moe.lib().moe_linear_w4(moe.moe_linear_shape(N, K, fmt, group, st), at(codes), at(scales), at(zeros), 1.0,
                                   at(x), xt, ldx, T, at(y), yt, ldy, flags, None, None)


@pytest.mark.parametrize("bad", [
    dict(N=0), dict(N=(1 << 24) + 1), dict(K=0), dict(K=48, ldx=48), dict(K=-32), dict(K=(1 << 17) + 32, ldx=1 << 18),
    dict(fmt=0), dict(fmt=4), dict(group=16), dict(group=0), dict(group=256), dict(st=3), dict(st=-1),
    dict(fmt=1, group=16), dict(fmt=2, group=32), dict(fmt=1, group=32, zeros=0), dict(T=-1), dict(T=(1 << 20) + 1),
    dict(xt=0), dict(xt=3), dict(yt=2), dict(yt=3), dict(flags=4), dict(N=15, flags=1), dict(codes=None),
    dict(scales=None), dict(x=None), dict(y=None), dict(codes=8), dict(x=8), dict(scales=1), dict(st=0, scales=2),
    dict(y=2), dict(yt=1, y=1), dict(ldx=60), dict(ldx=68), dict(ldy=15), dict(ldy=7, flags=1),
])
def test_refusals(moe, bad):
    raw = np.zeros(4096, dtype=np.uint8)
    p = raw.ctypes.data + (-raw.ctypes.data) % 256
    assert _call(moe, p, **bad) == moe.MOE_ERR_INVALID_ARG
    assert moe.lib().moe_last_error()


def test_no_tokens_is_no_call(moe):
    assert moe.lib().moe_linear_w4(moe.moe_linear_shape(16, 64, 3, 32, 1), None, None, None, 1.0, None, 1, 64, 0, None,
                                   0, 16, 0, None, None) == moe.MOE_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls would launch on host pointers")
def test_valid_arguments_reach_the_device(moe):
    raw = np.zeros(4096, dtype=np.uint8)
    p = raw.ctypes.data + (-raw.ctypes.data) % 256
    for kw in (dict(), dict(flags=3), dict(fmt=1), dict(fmt=2, group=16), dict(zeros=5), dict(yt=1, y=2), dict(xt=2, yt=2)):
        assert _call(moe, p, **kw) == moe.MOE_ERR_CUDA


def test_binding_refuses_what_the_library_cannot_see(moe):
    c = torch.zeros((16, 32), dtype=torch.uint8)
    s = torch.ones((16, 2), dtype=torch.bfloat16)
    with pytest.raises(ValueError):                                    # not CUDA tensors
        moe.moe_linear_w4(torch.zeros((1, 64), dtype=torch.bfloat16), c, s, torch.zeros((1, 16)), group=32)
    with pytest.raises(KeyError):
        moe.moe_linear_w4(torch.zeros((1, 64), dtype=torch.bfloat16), c, s, torch.zeros((1, 16)), fmt="bf16")
