"""Helpers of the block operators' GPU tests: guarded output buffers, and the formats in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

DEV = "cuda"
GUARD = 4096  # sentinel bytes before and after a guarded buffer
SENTINEL = 0xA5


class Guarded:
    """Output buffers inside sentinel bytes; check() asserts that none of those were written."""

    def __init__(self):
        self.bufs = []

    def __call__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((n + 2 * GUARD,), SENTINEL, dtype=torch.uint8, device=DEV)
        self.bufs.append(buf)
        return buf[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for buf in self.bufs:
            assert bool((buf[:GUARD] == SENTINEL).all()), "bytes before an output were written"
            assert bool((buf[-GUARD:] == SENTINEL).all()), "bytes after an output were written"


def bits(v):
    """float tensor -> bf16 bit patterns (torch.int16)."""
    return torch.as_tensor(v).to(torch.bfloat16).view(torch.int16)


def f64(b16):
    """bf16 bit patterns -> float64 on the CPU."""
    return b16.cpu().view(torch.bfloat16).double()


def e4m3(codes):
    """E4M3FN codes -> float64 on the CPU."""
    return codes.cpu().view(torch.float8_e4m3fn).double()


def rng(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float32)


def weights64(wdtype, w, s):
    """One weight matrix [rows, cols] of a format in float64, decoded from its definition."""
    if wdtype == "bf16":
        return w.view(torch.bfloat16).double()
    if wdtype == "fp8":
        v = w.view(torch.float8_e4m3fn).double()
        return v * s.double().repeat_interleave(128, 0)[:v.shape[0]].repeat_interleave(128, 1)
    e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                        dtype=torch.float64, device=w.device)
    v = torch.stack([e2m1[(w & 15).long()], e2m1[(w >> 4).long()]], -1).flatten(-2)
    return v * torch.exp2(s.double() - 127).repeat_interleave(32, 1)


def expert64(ew, e, x):
    """(g, u, bound, y, ybound) of one expert on rows x (float64): the projections' values, and the
    sums of absolute products behind them."""
    pick = lambda t: None if t is None else t[e]  # noqa: E731
    wg = weights64(ew.wdtype, ew.gate[e], pick(ew.s_gate))
    wu = weights64(ew.wdtype, ew.up[e], pick(ew.s_up))
    return x @ wg.T, x @ wu.T, x.abs() @ wg.abs().T, x.abs() @ wu.abs().T


def layer64(layer, ids, wts):
    """(out, error bound) of a synth.Layer in float64 for the routing ids, wts [T, k].  The bound takes
    sums of n fp32 terms as off by n * 2^-23 * sum|terms| (any order, products of scaled blocks rounded
    too), with MXFP4 weights a value of x as off by 2^-21 of its 128-block's largest, SiLU * up as 2^-18 (1 + |g|) relative (exp, its argument, and the reciprocal), w * h
    kept in two bf16 values as 2^-15; bf16's half step of the output (2^-8) comes on top."""
    dev = layer.x.device
    x = layer.x.view(torch.bfloat16).double()
    out = torch.zeros((layer.T, layer.H), dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    per = [(layer.experts, e, None) for e in sorted(set(ids.flatten().tolist()))]
    per += [(layer.shared, 0, "all")] if layer.shared is not None else []
    n_terms = (len(per) * layer.I)
    for ew, e, who in per:
        if who == "all":
            t, w = torch.arange(layer.T), torch.ones(layer.T, dtype=torch.float64)
        else:
            t, j = torch.nonzero(ids == e, as_tuple=True)
            w = wts[t, j].double()
        t, w = t.to(dev), w.to(dev)[:, None]
        g, u, ag, au = expert64(ew, e, x[t])
        h = g * torch.sigmoid(g) * u
        dg, du = layer.H * 2.0 ** -23 * ag, layer.H * 2.0 ** -23 * au
        if ew.wdtype == "mxfp4":
            top = x[t].abs().unflatten(1, (-1, 128)).amax(2).repeat_interleave(128, 1)
            more = expert64(ew, e, 2.0 ** -21 * top)
            dg, du = dg + more[2], du + more[3]
        dh = 1.1 * (u.abs() + du) * dg + (g * torch.sigmoid(g)).abs() * du + h.abs() * (2.0 ** -15 + 2.0 ** -18 * (1 + g.abs()))
        wd = weights64(ew.wdtype, ew.down[e], None if ew.s_down is None else ew.s_down[e])
        out[t] += (w * h) @ wd.T
        tol[t] += (w * dh) @ wd.abs().T + n_terms * 2.0 ** -23 * ((w * h).abs() @ wd.abs().T)
    return out, tol
