"""moe_router_scores against the product in 64 bits.

Tolerances.  Products of bf16 values (and of a bf16 value with each bf16 part of an fp32 weight) are
exact in fp32; a sum of n terms in fp32, in any order, is off by at most n * 2^-24 * sum|terms| (the
bound holds with n = H, 3 H for the three parts of an fp32 weight).  Inputs that are small whole
numbers have exact sums in every order: there the scores are bit-exact.
"""
import pytest
import torch

import routed_expert_grouped_amd as moe
from block_util import DEV, Guarded, bits, f64, randn, rng

pytestmark = pytest.mark.gpu

SIZES = [  # T, H, E: both kernels, ragged tiles, K tails, split and unsplit
    (1, 8, 1), (1, 7168, 256), (2, 256, 7), (3, 520, 16), (4, 1024, 64), (5, 2048, 129), (8, 7168, 384),
    (9, 264, 33), (16, 7168, 256), (17, 7168, 256), (31, 8, 5), (64, 72, 130), (127, 512, 128),
    (128, 1032, 129), (129, 2048, 255), (333, 7168, 384), (1000, 640, 1024), (4096, 512, 256),
    # around and above the large batches' tiles: one and several K steps, none that is whole, a last one of one chunk, both widths
    (2048, 64, 256), (2049, 8, 5), (2047, 72, 130), (2048, 72, 130), (2100, 1032, 384), (2300, 120, 300),
    (2048, 7168, 256), (2177, 2056, 1000), (5000, 192, 256), (2200, 1160, 100), (2050, 4096, 192),
    (10000, 8, 5), (9500, 64, 33), (9473, 72, 16), (5000, 1160, 100), (3300, 4096, 192), (2432, 64, 256),
    (2560, 7168, 256),
]


def call(x, w, T, E):
    G = Guarded()
    out = moe.moe_router_scores(x.to(DEV), w.to(DEV), scores=G((T, E), torch.float32))
    G.check()
    return out.cpu().double()


@pytest.mark.parametrize("T,H,E", SIZES)
@pytest.mark.parametrize("f32", [False, True])
def test_against_the_product(T, H, E, f32):
    gen = rng(T * 7 + H + E)
    x = bits(randn(gen, T, H))
    w = randn(gen, E, H) * 0.02
    w = w if f32 else bits(w)
    got = call(x, w, T, E)
    xd, wd = f64(x), (w.double() if f32 else f64(w))
    tol = (3 if f32 else 1) * H * 2.0 ** -24 * (xd.abs() @ wd.abs().T)
    assert bool(((got - xd @ wd.T).abs() <= tol).all())


@pytest.mark.parametrize("T,H,E", SIZES)
@pytest.mark.parametrize("f32", [False, True])
def test_whole_numbers_are_exact(T, H, E, f32):
    gen = rng(T + H * 3 + E)
    x = torch.randint(-8, 9, (T, H), generator=gen)
    w = torch.randint(-8, 9, (E, H), generator=gen)  # |sum| <= 64 H <= 2^19
    got = call(bits(x.float()), w.float() if f32 else bits(w.float()), T, E)
    assert torch.equal(got, x.double() @ w.double().T)


@pytest.mark.parametrize("T", [1, 5, 16, 17, 300, 2500, 10000])
def test_every_bit_of_an_fp32_weight_counts(T):
    """Rows that pick one weight each return it bit for bit."""
    H, E = 256, 40
    gen = rng(T)
    w = randn(gen, E, H)
    pick = torch.randint(0, H, (T,), generator=gen)
    x = torch.zeros(T, H)
    x[torch.arange(T), pick] = 1.0
    assert torch.equal(call(bits(x), w, T, E), w[:, pick].T.double())


@pytest.mark.parametrize("T", [4, 16, 40, 2100, 9500])
def test_nan_and_infinity_stay_in_their_row_or_column(T):
    H, E = 328, 48
    gen = rng(T)
    x, w = bits(randn(gen, T, H)), randn(gen, E, H)
    clean = call(x, w, T, E)
    x[2, 7] = 0x7FC0
    w[5, 300] = float("inf")
    got = call(x, w, T, E)
    rows, cols = torch.arange(T) != 2, torch.arange(E) != 5
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols])
    assert bool(torch.isnan(got[2]).all())
    sign = torch.sign(f64(x)[rows, 300])
    assert torch.equal(got[rows, 5], sign * float("inf"))


@pytest.mark.parametrize("T", [5, 40, 2100, 9500])
def test_fp32_weights_of_every_kind(T):
    """Weights of both signs down to 2^-100, infinities and NaNs of any payload: rows that pick one return it."""
    H, E = 128, 16
    gen = rng(T)
    w = randn(gen, E, H) * torch.exp2(torch.randint(-100, 100, (E, H), generator=gen).float())
    pick = torch.randint(0, H, (T,), generator=gen)
    x = torch.zeros(T, H)
    x[torch.arange(T), pick] = 1.0
    assert torch.equal(call(bits(x), w, T, E), w[:, pick].T.double())
    w[0, 3], w[1, 5], w[2, 7] = float("inf"), float("-inf"), float("nan")
    w.view(torch.int32)[3, 9] = 0x7F800001  # a NaN whose upper half is an infinity's
    x = torch.ones(T, H)
    got = call(bits(x), w, T, E)
    assert bool((got[:, 0] == float("inf")).all() and (got[:, 1] == float("-inf")).all())
    assert bool(torch.isnan(got[:, 2:4]).all() and torch.isfinite(got[:, 4:]).all())


def test_sums_in_the_same_order_every_time():
    gen = rng(1)
    x, w = bits(randn(gen, 700, 7168)).to(DEV), bits(randn(gen, 256, 7168)).to(DEV)
    a = moe.moe_router_scores(x, w).clone()
    for _ in range(3):
        assert torch.equal(moe.moe_router_scores(x, w), a)


def test_workspace_rules():
    assert moe.moe_router_scores_workspace_size(16, 7168, 256) == 0
    need = moe.moe_router_scores_workspace_size(17, 7168, 256)
    assert need > 0
    gen = rng(2)
    x, w = bits(randn(gen, 17, 7168)).to(DEV), bits(randn(gen, 256, 7168)).to(DEV)
    with pytest.raises(moe.MoeError) as e:
        moe.moe_router_scores(x, w, ws=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    assert e.value.status == moe.MOE_ERR_WORKSPACE
    G = Guarded()
    a = moe.moe_router_scores(x, w, ws=G((need,), torch.uint8)).clone()
    G.check()
    assert torch.equal(a, moe.moe_router_scores(x, w))


def test_no_tokens():
    x = torch.empty((0, 256), dtype=torch.int16, device=DEV)
    w = torch.zeros((8, 256), dtype=torch.int16, device=DEV)
    assert moe.moe_router_scores(x, w).shape == (0, 8)


@pytest.mark.parametrize("T", [3, 200, 2048, 2500])
def test_streams_and_graph(T):
    gen = rng(T)
    x, w = bits(randn(gen, T, 2048)).to(DEV), bits(randn(gen, 256, 2048)).to(DEV)
    want = moe.moe_router_scores(x, w).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_router_scores(x, w, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    ws = torch.empty(max(16, moe.moe_router_scores_workspace_size(T, 2048, 256)), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_router_scores(x, w, scores=out, ws=ws)
    for rep in range(4):
        if rep == 3:
            x.copy_(torch.roll(x, 1, 0))
            want = moe.moe_router_scores(x, w).clone()
        out.zero_()
        ws.fill_(255)  # NaN patterns: nothing of an earlier replay is read
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_binding_refuses_other_layouts():
    x = torch.zeros((8, 256), dtype=torch.int16, device=DEV)
    w = torch.zeros((16, 256), dtype=torch.int16, device=DEV)
    for a, b, kw in ((x.t(), w, {}), (x, w[:, :128], {}), (x, w.cpu(), {}), (x.float(), w, {}),
                     (x, w.half(), {}), (x[0], w, {}), (x, w[:, ::2], {}),
                     (x, w, dict(scores=torch.empty((8, 15), device=DEV)))):
        with pytest.raises(ValueError):
            moe.moe_router_scores(a, b, **kw)
