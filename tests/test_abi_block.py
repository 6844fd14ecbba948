"""The block operators' argument checks, on the host before anything is enqueued (no GPU needed)."""
import ctypes
import os

import pytest
import torch

import routed_expert_grouped_amd as moe

pytestmark = [pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="libmoe.so not built"),
              # fake device pointers: run only where no GPU is visible
              pytest.mark.skipif(torch.cuda.device_count() > 0, reason="needs a host without a GPU")]

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1008)
OK, INV, UNS, WSP = moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


def norm(x=FAKE, res=FAKE, w=FAKE, rows=4, K=256, eps=1e-6, s=FAKE, y=FAKE, c=FAKE, e=FAKE, pitch=16):
    return moe.lib().moe_rmsnorm_quantize_act(x, res, w, rows, K, eps, s, y, c, e, pitch, None)


def test_norm():
    assert norm(rows=0) == OK
    assert norm(rows=0, x=None, w=None, y=None, s=None, c=None, e=None) == OK
    for bad in (dict(x=None), dict(w=None), dict(rows=-1), dict(K=0), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(c=None), dict(e=None),
                dict(pitch=1), dict(y=None, c=None, e=None), dict(res=None), dict(x=ODD), dict(res=ODD),
                dict(w=ODD), dict(s=ODD), dict(y=ODD), dict(c=ODD), dict(e=ODD)):
        assert norm(**bad) == INV, bad
    for bad in (dict(K=100), dict(K=200), dict(K=16384 + 128), dict(K=12, c=None, e=None)):
        assert norm(**bad) == UNS, bad


def router(x=FAKE, T=100, H=256, w=FAKE, dt=0, E=64, out=FAKE, ws=FAKE, n=1 << 30):
    return moe.lib().moe_router_scores(x, T, H, w, dt, E, out, ws, n, None)


def test_router():
    assert router(T=0) == OK and router(T=0, x=None, w=None, out=None, ws=None) == OK
    for bad in (dict(x=None), dict(w=None), dict(out=None), dict(T=-1), dict(H=0), dict(E=0), dict(dt=2),
                dict(dt=-1), dict(x=ODD), dict(w=ODD), dict(out=ODD)):
        assert router(**bad) == INV, bad
    for bad in (dict(H=100), dict(H=16384 + 8), dict(E=1025), dict(T=1 << 24, E=1024),
                dict(T=(1 << 31) - 1, H=8, E=1)):
        assert router(**bad) == UNS, bad
    need = moe.moe_router_scores_workspace_size(100, 7168, 64)
    assert need % (100 * 64 * 4) == 0 and need > 0
    assert router(H=7168, ws=None) == WSP and router(H=7168, n=need - 1) == WSP
    assert router(H=7168, ws=ODD) == INV
    size = moe.lib().moe_router_scores_workspace_size
    n = ctypes.c_size_t(1)
    assert size(100, 7168, 64, None) == INV and size(-1, 7168, 64, ctypes.byref(n)) == INV
    assert size(100, 7, 64, ctypes.byref(n)) == UNS
    assert size(0, 7168, 64, ctypes.byref(n)) == OK and n.value == 0


def weights(dtype=0, n=4, H=256, I=128, ptr=FAKE, scales=True):
    s = ptr.value if scales else None
    return moe.MoeExpertWeights(dtype, n, H, I, ptr.value, ptr.value, ptr.value, s, s, s)


def few(scores=FAKE, x=FAKE, T=4, k=2, fn=0, w=None, sh=None, ids=FAKE, tw=FAKE, out=FAKE, ws=FAKE, n=1 << 30):
    w = weights() if w is None else w
    return moe.lib().moe_layer_few(scores, x, T, k, fn, 1, ctypes.byref(w),
                                   None if sh is None else ctypes.byref(sh), ids, tw, out, ws, n, None)


def test_layer_few():
    assert few(T=0) == OK and few(T=0, scores=None, x=None, ids=None, tw=None, out=None, ws=None) == OK
    one = lambda **kw: weights(**(dict(n=1) | kw))  # noqa: E731
    assert few(T=0, sh=one()) == OK
    for bad in (dict(scores=None), dict(x=None), dict(ids=None), dict(tw=None), dict(out=None), dict(T=-1),
                dict(k=0), dict(k=5), dict(fn=2), dict(scores=ODD), dict(x=ODD), dict(ids=ODD), dict(tw=ODD),
                dict(out=ODD), dict(ws=ODD), dict(w=weights(dtype=3)), dict(w=weights(scales=False)),
                dict(w=weights(ptr=ODD)), dict(sh=weights()), dict(sh=one(dtype=1)), dict(sh=one(H=128)),
                dict(sh=one(I=256)), dict(sh=one(ptr=ODD))):
        assert few(**bad) == INV, bad
    for bad in (dict(T=9), dict(w=weights(H=200)), dict(w=weights(I=64)), dict(w=weights(n=1025)),
                dict(w=weights(n=64), k=33), dict(w=weights(H=16384), T=4), dict(w=weights(H=7296), T=8)):
        assert few(**bad) == UNS, bad
    w = weights()
    need = moe.moe_layer_few_workspace_size(4, 2, w)
    assert need >= (4 + 1) * 2 * 4 * 128 * 2
    assert few(ws=None) == WSP and few(n=need - 1) == WSP
    assert moe.moe_layer_few_workspace_size(0, 2, w) == 0
    n = ctypes.c_size_t(0)
    size = moe.lib().moe_layer_few_workspace_size
    assert size(4, 2, ctypes.byref(w), None) == INV and size(4, 2, None, ctypes.byref(n)) == INV
    assert size(9, 2, ctypes.byref(w), ctypes.byref(n)) == UNS
    assert size(3, 2, ctypes.byref(weights(H=16384)), ctypes.byref(n)) == OK


def linear(a=FAKE, e=FAKE, pitch=16, M=4, N=100, K=256, w=FAKE, s=FAKE, y=FAKE):
    return moe.lib().moe_linear_a8(a, e, pitch, M, N, K, w, s, y, None)


def test_linear():
    assert linear(M=0) == OK and linear(M=0, a=None, e=None, w=None, s=None, y=None) == OK
    for bad in (dict(a=None), dict(e=None), dict(w=None), dict(s=None), dict(y=None), dict(M=-1), dict(N=0),
                dict(K=0), dict(pitch=1), dict(a=ODD), dict(e=ODD), dict(w=ODD), dict(s=ODD), dict(y=ODD)):
        assert linear(**bad) == INV, bad
    for bad in (dict(K=100), dict(K=65536 + 128, pitch=1024), dict(M=1 << 30, N=1 << 20),
                dict(M=(1 << 31) - 1, N=1 << 20), dict(M=1 << 20, N=(1 << 31) - 1),
                dict(M=(1 << 31) - 1, N=(1 << 31) - 1), dict(M=1, N=(1 << 31) - 1)):
        assert linear(**bad) == UNS, bad


def test_binding_needs_gpu_tensors():
    x, g = torch.zeros((4, 256), dtype=torch.int16), torch.zeros(256, dtype=torch.int16)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm_quantize_act(x, g)
    with pytest.raises(ValueError):
        moe.moe_router_scores(x, x)
