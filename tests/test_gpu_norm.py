"""moe_rmsnorm_quantize_act against the formula in 64 bits.

Tolerances.  sum: bit-exact (an fp32 sum of two bf16 values rounded to bf16, as torch does it).  v is
computed in double and rounded to fp32 (2^-24), then y to bf16 (half a step, 2^-8 of the value):
|y - v| <= (2^-8 + 2^-22) |v|.  The exponent is the smallest with max|v| <= 448 * 2^e, up to v's own fp32
rounding, and a code is half an E4M3 step off: 2^-4 of the value, or 2^-10 * 2^e below 2^-6 * 2^e.
"""
import pytest
import torch

import routed_expert_grouped_amd as moe
from block_util import DEV, Guarded, bits, e4m3, f64, randn, rng

pytestmark = pytest.mark.gpu

EPS = 1e-6


def reference(x, res, g, eps=EPS):
    """(bf16 bits of the sum, v in float64)."""
    s = x if res is None else bits(x.view(torch.bfloat16).float() + res.view(torch.bfloat16).float())
    d = f64(s)
    return s, d / torch.sqrt(d.square().mean(-1, keepdim=True) + eps) * f64(g)


def check_codes(codes, exps, v):
    rows, K = v.shape
    blk = v.reshape(rows, K // 128, 128)
    e = exps.cpu()[:, :K // 128].double()
    amax = blk.abs().amax(-1)
    lim = 448.0 * torch.exp2(e)
    zero = amax == 0
    assert bool((e[zero] == 0).all())
    assert bool((amax <= lim * (1 + 2.0 ** -23)).all())
    small = (e > -127) & ~zero
    assert bool((amax[small] >= 0.5 * lim[small] * (1 - 2.0 ** -23)).all())
    got = e4m3(codes).reshape(blk.shape)
    want = blk / torch.exp2(e)[..., None]
    tol = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64)) * (1 + 2.0 ** -20)
    assert bool(((got - want).abs() <= tol).all())
    assert bool((torch.signbit(got) == torch.signbit(want))[want != 0].all())


def run(x, res, g, normed=True, quantized=True, pitch=None, eps=EPS):
    rows, K = x.shape
    G = Guarded()
    out = dict(sum_out=G(x.shape, torch.int16) if res is not None else None,
               y=G(x.shape, torch.int16) if normed else None,
               codes=G(x.shape, torch.uint8) if quantized else None,
               exps=G((rows, pitch or moe.exp_pitch(K)), torch.int8) if quantized else None)
    got = moe.moe_rmsnorm_quantize_act(x.to(DEV), g.to(DEV), None if res is None else res.to(DEV), eps,
                                       normed, quantized, **out)
    G.check()
    return got


def inputs(rows, K, seed, residual=True):
    gen = rng(seed)
    x = bits(randn(gen, rows, K))
    res = bits(4.0 * randn(gen, rows, K)) if residual else None
    return x, res, bits(1.0 + 0.1 * randn(gen, K))


@pytest.mark.parametrize("rows,K", [(1, 128), (1, 7168), (3, 256), (5, 384), (7, 4096), (2, 4224), (33, 2048),
                                    (4, 8192), (3, 8320), (2, 16384), (300, 512), (1000, 1152)])
@pytest.mark.parametrize("residual", [False, True])
def test_all_outputs(rows, K, residual):
    x, res, g = inputs(rows, K, rows * 131 + K, residual)
    total, y, codes, exps = run(x, res, g)
    s, v = reference(x, res, g)
    if residual:
        assert torch.equal(total.cpu(), s)
    else:
        assert total is None
    assert bool(((f64(y) - v).abs() <= (2.0 ** -8 + 2.0 ** -22) * v.abs()).all())
    check_codes(codes, exps, v)
    # the padding of an exponent row is left as it was
    assert bool((exps.cpu()[:, K // 128:].view(torch.uint8) == 0xA5).all())


@pytest.mark.parametrize("K", [8, 16, 72, 520, 1000, 7160, 16376])
def test_odd_widths_without_codes(K):
    x, res, g = inputs(9, K, K)
    total, y, codes, exps = run(x, res, g, quantized=False)
    assert codes is None and exps is None
    s, v = reference(x, res, g)
    assert torch.equal(total.cpu(), s)
    assert bool(((f64(y) - v).abs() <= (2.0 ** -8 + 2.0 ** -22) * v.abs()).all())


def test_codes_alone_and_unpadded_exponents():
    x, res, g = inputs(37, 640, 1, residual=False)
    total, y, codes, exps = run(x, None, g, normed=False, pitch=5)
    assert total is None and y is None and exps.shape == (37, 5)
    check_codes(codes, exps, reference(x, None, g)[1])


def test_without_a_stored_sum():
    x, res, g = inputs(5, 512, 2)
    y = torch.empty((5, 512), dtype=torch.int16, device=DEV)
    dx, dr, dg = x.to(DEV), res.to(DEV), g.to(DEV)  # (held until the call has run)
    st = moe.lib().moe_rmsnorm_quantize_act(moe._p(dx), moe._p(dr), moe._p(dg), 5, 512, EPS, None,
                                            moe._p(y), None, None, 0, moe._s(None))
    assert st == moe.MOE_OK
    v = reference(x, res, g)[1]
    assert bool(((f64(y) - v).abs() <= (2.0 ** -8 + 2.0 ** -22) * v.abs()).all())


def test_residual_updated_in_place():
    """sum_out may be the residual or x: the same outputs as with a buffer of its own."""
    x, res, g = (t.to(DEV) for t in inputs(50, 7168, 3))
    want = [t.clone() for t in moe.moe_rmsnorm_quantize_act(x, g, res)]
    for which in ("residual", "x"):
        xx, rr = x.clone(), res.clone()
        got = moe.moe_rmsnorm_quantize_act(xx, g, rr, sum_out=rr if which == "residual" else xx)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        assert torch.equal(rr if which == "residual" else xx, want[0])


def test_magnitudes_zero_rows_and_cancelling_sums():
    """Rows from bf16's subnormals to 1e38 (their squares pass fp32's range on both sides), a row of
    zeros, a residual that cancels x, signed zeros, a block of zeros beside a full one."""
    K = 512
    gen = rng(4)
    mags = [2.0 ** p for p in (-133, -126, -80, -40, 0, 40, 80, 120, 126)]
    x = torch.cat([bits(randn(gen, 1, K).clamp(-1.9, 1.9) * m) for m in mags] + [torch.zeros((4, K), dtype=torch.int16)])
    res = torch.zeros_like(x)
    res[-4] = 0                                     # zeros
    x[-3] = bits(randn(gen, K)); res[-3] = x[-3] ^ -32768   # cancels exactly
    x[-2] = -32768                                  # -0
    x[-1, 128:256] = bits(randn(gen, 128))          # one block of four
    g = bits(1.0 + 0.1 * randn(gen, K))
    total, y, codes, exps = run(x, res, g)
    s, v = reference(x, res, g)
    assert torch.equal(total.cpu() & 0x7FFF, s & 0x7FFF)
    got = f64(y)
    # below bf16's normals a half step is 2^-134
    assert bool(((got - v).abs() <= (2.0 ** -8 + 2.0 ** -22) * v.abs() + 2.0 ** -134).all())
    check_codes(codes, exps, v)
    assert bool((got[-4:-1] == 0).all()) and bool((got[-1, :128] == 0).all())


def test_large_weights_reach_the_exponent_clamp():
    K = 256
    gen = rng(5)
    x = bits(randn(gen, 3, K))
    g = bits(torch.full((K,), 2.0 ** -125))
    _, _, codes, exps = run(x, None, g)
    check_codes(codes, exps, reference(x, None, g)[1])
    assert int(exps.cpu()[:, :2].min()) == -127
    g = bits(torch.full((K,), 2.0 ** 120))
    _, _, codes, exps = run(x, None, g)
    check_codes(codes, exps, reference(x, None, g)[1])


def test_nan_and_infinity_stay_in_their_rows():
    x, res, g = inputs(6, 384, 6)
    clean = run(x, res, g)
    x2 = x.clone()
    x2[1, 200] = 0x7FC0   # NaN
    x2[3, 5] = 0x7F80     # inf
    total, y, codes, exps = run(x2, res, g)
    keep = [0, 2, 4, 5]
    for a, b in zip(clean, (total, y, codes, exps)):
        assert torch.equal(a.cpu()[keep], b.cpu()[keep])
    assert bool(torch.isnan(f64(y)[1]).all()) and bool(torch.isnan(e4m3(codes)[1]).all())
    row = f64(y)[3]
    assert bool(torch.isnan(row[5])) and bool((row[torch.arange(384) != 5] == 0).all())
    assert bool(torch.isnan(e4m3(codes)[3, 5]))
    assert bool((exps.cpu()[[1, 3], :3] == 0).all())


def test_many_rows():
    """More rows than a launch has workgroups of this size resident, in two widths."""
    for rows, K in ((20000, 128), (4096, 2048)):
        x, res, g = inputs(rows, K, rows)
        total, y, codes, exps = run(x, res, g)
        s, v = reference(x, res, g)
        assert torch.equal(total.cpu(), s)
        assert bool(((f64(y) - v).abs() <= (2.0 ** -8 + 2.0 ** -22) * v.abs()).all())
        check_codes(codes, exps, v)


def test_no_rows():
    x = torch.empty((0, 256), dtype=torch.int16, device=DEV)
    g = torch.zeros(256, dtype=torch.int16, device=DEV)
    out = moe.moe_rmsnorm_quantize_act(x, g, x)
    assert [t.shape[0] for t in out] == [0, 0, 0, 0]


def test_streams_and_graph():
    """On a side stream, and captured: each replay equals the eager call, also after new inputs."""
    x, res, g = (t.to(DEV) for t in inputs(17, 7168, 8))
    want = [t.clone() for t in moe.moe_rmsnorm_quantize_act(x, g, res)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_rmsnorm_quantize_act(x, g, res, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[:, :56], b[:, :56])
    bufs = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_rmsnorm_quantize_act(x, g, res, sum_out=bufs[0], y=bufs[1], codes=bufs[2], exps=bufs[3])
    for rep in range(4):
        if rep == 3:
            x.copy_(torch.roll(x, 1, 0))
            want = [t.clone() for t in moe.moe_rmsnorm_quantize_act(x, g, res)]
        for b in bufs:
            b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(bufs, want):
            assert torch.equal(a[:, :56], b[:, :56])


def test_binding_refuses_other_layouts():
    x, res, g = (t.to(DEV) for t in inputs(8, 256, 9))
    call = moe.moe_rmsnorm_quantize_act
    for bad in (dict(x=x.t()), dict(x=x.view(torch.float16)), dict(weight=g[:128]), dict(residual=res[:4]),
                dict(residual=res.cpu()), dict(residual=None, sum_out=x), dict(codes=x),
                dict(exps=torch.empty((8, 1), dtype=torch.int32, device=DEV)), dict(x=x[:, :128])):
        kw = dict(x=x, weight=g, residual=res) | bad
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(moe.MoeError):
        call(x, g, res, eps=0.0)
    with pytest.raises(moe.MoeError):
        call(x, g, res, pitch=1)
