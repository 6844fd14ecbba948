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
