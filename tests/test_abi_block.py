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
    for bad in (dict(H=100), dict(H=16384 + 8), dict(E=1025), dict(T=1 << 24, E=1024)):
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


def test_binding_needs_gpu_tensors():
    x, g = torch.zeros((4, 256), dtype=torch.int16), torch.zeros(256, dtype=torch.int16)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm_quantize_act(x, g)
    with pytest.raises(ValueError):
        moe.moe_router_scores(x, x)
