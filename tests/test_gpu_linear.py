"""moe_linear_a8 against the product in 64 bits.

Tolerances.  Products of two E4M3 values are exact in fp32, and so is a power of two on them.  A sum of n
fp32 terms in any order (and with truncating adds inside the matrix instruction) is off by at most
n * 2^-23 * sum|terms|, with K products and two roundings a block; the output's bf16 rounding adds
half a step, 2^-8 of the value.  Whole-number inputs have exact sums: there the output is the exact
sum rounded to bf16, bit for bit.
"""
import pytest
import torch

import routed_expert_grouped_amd as moe
from block_util import DEV, Guarded, bits, e4m3, randn, rng

pytestmark = pytest.mark.gpu

SIZES = [  # M, N, K
    (1, 1, 128), (1, 2048, 7168), (2, 7, 256), (15, 16, 384), (16, 17, 1152), (17, 100, 1024), (31, 128, 128),
    (32, 129, 2048), (33, 576, 512), (64, 200, 7168), (65, 64, 1280), (200, 1000, 896), (256, 130, 640),
    (257, 127, 384), (300, 2112, 256), (513, 129, 1152), (1000, 1000, 128), (3, 5, 65536), (129, 48, 18432),
    (300, 40, 16512),
    (3585, 3400, 256), (4000, 3333, 384),  # 256 x 256 tiles, ragged both ways
    (3500, 3500, 2304),                    # ... and more than one window of scales
    # 128 x 128 tiles, at most one a CU (1, 2, 3, 5 and 18 K steps) and two
    (1100, 300, 128), (1030, 129, 256), (1100, 3000, 384), (1500, 700, 640), (1026, 200, 2304),
    (1300, 3333, 1152), (2000, 2500, 128), (1025, 4200, 2304),
]


def quantised(gen, M, K):
    codes = (randn(gen, M, K) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, torch.randint(-9, 3, (M, K // 128), generator=gen, dtype=torch.int8)


def weights(gen, N, K):
    w = (randn(gen, N, K) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return w, torch.rand((-(-N // 128), K // 128), generator=gen) * 2e-4 + 1e-4


def padded(exps, pitch=None, fill=77):
    M, kb = exps.shape
    out = torch.full((M, pitch or moe.exp_pitch(128 * kb)), fill, dtype=torch.int8)
    out[:, :kb] = exps
    return out


def call(codes, exps, w, s):
    G = Guarded()
    y = moe.moe_linear_a8(codes.to(DEV), exps.to(DEV), w.to(DEV), s.to(DEV),
                          y=G((codes.shape[0], w.shape[0]), torch.int16))
    G.check()
    return y


def dense(codes, exps, w, s):
    """x and W in float64, on the GPU."""
    kb = w.shape[1] // 128
    x = e4m3(codes).to(DEV) * torch.exp2(exps[:, :kb].double()).to(DEV).repeat_interleave(128, 1)
    W = e4m3(w).to(DEV) * s.double().to(DEV).repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)
    return x, W


def check(codes, exps, w, s):
    got = call(codes, exps, w, s).view(torch.bfloat16).double()
    x, W = dense(codes, exps, w, s)
    ref = x @ W.T
    K = w.shape[1]
    tol = (K + K // 64) * 2.0 ** -23 * (x.abs() @ W.abs().T)
    assert bool(((got - ref).abs() <= 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * tol).all())


@pytest.mark.parametrize("M,N,K", SIZES)
def test_against_the_product(M, N, K):
    gen = rng(M + 3 * N + K)
    codes, exps = quantised(gen, M, K)
    w, s = weights(gen, N, K)
    check(codes, padded(exps), w, s)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_whole_numbers_are_exact(M, N, K):
    gen = rng(M * 5 + N + K)
    hi = 5 if K > 20000 else 8  # |sum| <= hi^2 K * 2 < 2^24
    x = torch.randint(-hi, hi + 1, (M, K), generator=gen)
    w = torch.randint(-hi, hi + 1, (N, K), generator=gen)
    if K <= 20000:
        w[w.abs() > 3] = 1
    s = torch.exp2(torch.randint(0, 2, (-(-N // 128), K // 128), generator=gen).float())
    e = torch.randint(-1, 1, (M, K // 128), generator=gen, dtype=torch.int8)
    f8 = lambda t: t.float().to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    got = call(f8(x), padded(e), f8(w), s)
    a, b = dense(f8(x), e, f8(w), s)
    assert torch.equal(got.cpu(), bits((a @ b.T).float().cpu()))


@pytest.mark.parametrize("M", [3, 20, 100, 300])
def test_any_exponent_pitch(M):
    gen = rng(M)
    codes, exps = quantised(gen, M, 640)
    w, s = weights(gen, 72, 640)
    want = call(codes, padded(exps), w, s)
    for pitch in (5, 6, 7, 31):
        assert torch.equal(call(codes, padded(exps, pitch), w, s), want)


@pytest.mark.parametrize("M", [3, 300])
def test_extreme_scales(M):
    """Zero, subnormal, huge and negative weight scales beside ordinary ones, block exponents at both ends."""
    gen = rng(M)
    K, N = 1024, 256
    codes, exps = quantised(gen, M, K)
    w, s = weights(gen, N, K)
    s[0] = torch.tensor([0.0, 1e-40, 1e-4, 1e-38, 1e20, -1e-4, 0.0, 1e-45])
    exps[:, 4] = -100  # beside the 1e20 scale
    check(codes, padded(exps), w, s)
    s2 = torch.full((2, 8), 1.0)
    e2 = torch.zeros_like(exps)
    e2[:, ::2] = -127
    check(codes, padded(e2), w, s2)
    small = (codes & 0x8F)  # subnormal codes and zeros: 2^-9 .. 7 * 2^-9
    e2[:] = 100
    check(small, padded(e2), w, s2 * 2.0 ** -60)


@pytest.mark.parametrize("M", [5, 40, 300])
def test_nan_stays_in_its_row_and_column(M):
    gen = rng(M)
    codes, exps = quantised(gen, M, 512)
    w, s = weights(gen, 150, 512)
    clean = call(codes, padded(exps), w, s)
    codes[2, 300] = 0x7F
    w[9, 17] = 0xFF
    s[1, 0] = float("inf")  # outputs 128 on
    got = call(codes, padded(exps), w, s)
    rows, cols = torch.arange(M) != 2, (torch.arange(150) != 9) & (torch.arange(150) < 128)
    assert torch.equal(got.cpu()[rows][:, cols], clean.cpu()[rows][:, cols])
    f = got.view(torch.bfloat16).float()
    assert bool(torch.isnan(f[2]).all()) and bool(torch.isnan(f[:, 9]).all())
    assert not bool(torch.isfinite(f[:, 128:]).any())


def test_rows_agree_with_the_expert_call():
    """The grouped down projection with the identity grouping computes the same product."""
    gen = rng(1)
    M, N, K = 300, 512, 1024
    codes, exps = quantised(gen, M, K)
    w, s = weights(gen, N, K)
    a = call(codes, padded(exps), w, s).view(torch.bfloat16).double()
    dw, ds = w.to(DEV), s.to(DEV)
    W = moe.MoeExpertWeights(moe.MOE_W_FP8_E4M3_B128, 1, N, K, dw.data_ptr(), dw.data_ptr(), dw.data_ptr(),
                             ds.data_ptr(), ds.data_ptr(), ds.data_ptr())
    b = moe.moe_expert_down_a8(codes.to(DEV), padded(exps).to(DEV), M, 1, None, W).view(torch.bfloat16).double()
    assert float((a - b).norm() / b.norm()) <= 2.0 ** -8


def test_no_rows():
    gen = rng(2)
    w, s = weights(gen, 16, 256)
    y = moe.moe_linear_a8(torch.empty((0, 256), dtype=torch.uint8, device=DEV),
                          torch.empty((0, 16), dtype=torch.int8, device=DEV), w.to(DEV), s.to(DEV))
    assert y.shape == (0, 16)


@pytest.mark.parametrize("M", [4, 500])
def test_streams_and_graph(M):
    gen = rng(M)
    codes, exps = quantised(gen, M, 1024)
    w, s = weights(gen, 300, 1024)
    codes, exps, w, s = codes.to(DEV), padded(exps).to(DEV), w.to(DEV), s.to(DEV)
    want = moe.moe_linear_a8(codes, exps, w, s).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_linear_a8(codes, exps, w, s, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_linear_a8(codes, exps, w, s, y=out)
    for rep in range(4):
        if rep == 3:
            codes.copy_(torch.roll(codes, 1, 0))
            want = moe.moe_linear_a8(codes, exps, w, s).clone()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_binding_refuses_other_layouts():
    gen = rng(3)
    codes, exps = quantised(gen, 8, 512)
    w, s = weights(gen, 200, 512)
    ok = dict(codes=codes.to(DEV), exps=padded(exps).to(DEV), w=w.to(DEV), s_w=s.to(DEV))
    moe.moe_linear_a8(**ok)
    for bad in (dict(codes=ok["codes"].t()), dict(codes=ok["codes"].view(torch.int8)), dict(w=ok["w"][:, :256]),
                dict(exps=ok["exps"][:4]), dict(s_w=ok["s_w"][:1]), dict(s_w=ok["s_w"].double()), dict(w=w),
                dict(y=torch.empty((8, 201), dtype=torch.int16, device=DEV)), dict(codes=ok["codes"][0])):
        with pytest.raises(ValueError):
            moe.moe_linear_a8(**(ok | bad))
    with pytest.raises(moe.MoeError):
        moe.moe_linear_a8(**(ok | dict(exps=torch.zeros((8, 3), dtype=torch.int8, device=DEV))))
