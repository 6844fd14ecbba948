"""The calls around the layer and the layer together, as a transformer block runs them (MoeBlock): every stage of
one run against its formula in 64 bits on what the stage before stored, the block against the same calls made
one by one bit for bit, and captured into a graph; MoeLayer's two-launch form."""
import dataclasses

import pytest
import torch

import routed_expert_grouped_amd as moe
import synth
from block_util import DEV, bits, e4m3, expert64, f64, layer64, randn, rng, weights64

pytestmark = pytest.mark.gpu


def make(T, H, I, E, k, wdtype, seed, shared=True):
    cfg = dict(T=T, H=H, I=I, E=E, k=k, score_fn="sigmoid", renorm=1, scores="normal", wdtype=wdtype)
    layer = synth.make_layer(cfg, seed=seed).to(DEV)
    gen = rng(seed)
    inputs = dict(hidden=bits(randn(gen, T, H)).to(DEV), residual=bits(randn(gen, T, H)).to(DEV),
                  norm_w=bits(1 + 0.2 * randn(gen, H)).to(DEV),
                  router_w=(randn(gen, E, H) * 0.05).to(DEV))
    return (layer if shared else dataclasses.replace(layer, shared=None)), inputs


def block(layer, inp, **kw):
    return moe.MoeBlock(layer.T, layer.H, layer.I, layer.E, layer.k, inp["norm_w"], inp["router_w"],
                        layer.experts, layer.shared, **kw)


def check_front(B, inp, s):
    """The sum, the normed rows and the scores of a run, each from what the run stored before it."""
    want = f64(inp["hidden"]) + f64(inp["residual"])
    assert torch.equal(s.cpu(), bits(want.float()))  # (both have 8 bits: fp32 holds the sum, or rounds far below bf16)
    s64 = f64(s)
    n = s64 / (s64.square().mean(1, keepdim=True) + B.eps).sqrt() * f64(inp["norm_w"])
    got = f64(B.normed)
    # half a step of bf16, and the fp32 value between it and the formula
    assert bool(((got - n).abs() <= n.abs() * (2.0 ** -8 + 2.0 ** -22)).all())
    w = inp["router_w"].cpu().double()
    tol = 3 * B.H * 2.0 ** -24 * (got.abs() @ w.abs().T)
    assert bool(((B.scores.cpu().double() - got @ w.T).abs() <= tol).all())


@pytest.mark.parametrize("wdtype", ["fp8", "bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 5, 8])
def test_a_few_tokens(T, wdtype):
    layer, inp = make(T, 768, 384, 24, 4, wdtype, seed=T)
    B = block(layer, inp)
    assert B.layer.few
    out, s = B.forward(inp["hidden"], inp["residual"])
    torch.cuda.synchronize()
    check_front(B, inp, s)
    ids, wts = moe.moe_route(B.scores, layer.k)
    assert torch.equal(ids, B.layer.topk_ids) and torch.equal(wts, B.layer.topk_w)
    seen = dataclasses.replace(layer, x=B.normed, scores=B.scores)
    ref, tol = layer64(seen, ids.cpu(), wts.cpu())
    err = (out.view(torch.bfloat16).double() - ref).abs()
    assert bool((err <= ref.abs() * 2.0 ** -8 + (1 + 2.0 ** -8) * tol).all())


@pytest.mark.parametrize("T,few", [(8, False), (9, "auto"), (60, "auto"), (700, "auto")])
def test_the_separate_calls(T, few):
    """Above a few tokens (and where asked for) the block is MoeLayer's separate launches on the same scores."""
    layer, inp = make(T, 512, 256, 16, 3, "fp8", seed=T)
    B = block(layer, inp, few=few)
    assert not B.layer.few
    out, s = B.forward(inp["hidden"], inp["residual"])
    out = out.clone()
    check_front(B, inp, s)
    L = moe.MoeLayer(T, 512, 256, 16, 3, layer.experts, layer.shared)
    assert torch.equal(L.forward(B.scores, B.normed)[:T], out)


@pytest.mark.parametrize("wdtype", ["fp8", "mxfp4"])
@pytest.mark.parametrize("shared", [True, False])
def test_the_norms_codes_go_to_the_experts(wdtype, shared):
    T, H, I, E, k = 300, 512, 256, 8, 4
    layer, inp = make(T, H, I, E, k, wdtype, seed=7, shared=shared)
    B = block(layer, inp, act="fp8")
    assert B.codes is not None
    out, s = B.forward(inp["hidden"], inp["residual"])
    out = out.clone()
    torch.cuda.synchronize()
    check_front(B, inp, s)
    # the same calls one by one
    _, normed, codes, exps = moe.moe_rmsnorm_quantize_act(inp["hidden"], inp["norm_w"], inp["residual"])
    assert torch.equal(codes, B.codes) and torch.equal(exps[:, :H // 128], B.exps[:, :H // 128])
    ids, wts = moe.moe_route(moe.moe_router_scores(normed, inp["router_w"]), k)
    counts, offsets, perm, inv = moe.moe_permute(ids, E)[:4]
    w = moe.expert_weights(layer.experts)
    h = moe.moe_expert_gate_up_a8(codes, exps, k, perm, offsets, w)
    y = moe.moe_expert_down_a8(*moe.moe_quantize_act(h), T, k, offsets, w)
    sy = None
    if shared:
        ws = moe.expert_weights(layer.shared)
        sh = moe.moe_expert_gate_up_a8(codes, exps, 1, None, None, ws)
        sy = moe.moe_expert_down_a8(*moe.moe_quantize_act(sh), T, 1, None, ws)
    assert torch.equal(moe.moe_combine(y, inv, wts, sy, T, k, H), out)
    # and the formula on the codes: h is rounded to bf16 (2^-8) and to E4M3 (2^-4 of a value, or 2^-10 of
    # its block's 448th part where the code is subnormal), y and the shared output to bf16 each
    x = e4m3(codes) * torch.exp2(exps[:, :H // 128].cpu().double()).repeat_interleave(128, 1)
    ref, tol = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    experts = layer.experts.to("cpu")
    per = [(experts, e) for e in range(E)] + ([(layer.shared.to("cpu"), None)] if shared else [])
    for ew, e in per:
        if e is None:
            t, g = torch.arange(T), torch.ones(T, 1, dtype=torch.float64)
        else:
            t, j = torch.nonzero(ids.cpu() == e, as_tuple=True)
            g = wts.cpu()[t, j].double()[:, None]
        gate, up, ag, au = expert64(ew, e or 0, x[t])
        act = gate * torch.sigmoid(gate)
        hv = act * up
        dg, du = H * 2.0 ** -23 * ag, H * 2.0 ** -23 * au
        dh = 1.1 * (up.abs() + du) * dg + act.abs() * du + hv.abs() * 2.0 ** -15
        top = hv.abs().unflatten(1, (-1, 128)).amax(2).repeat_interleave(128, 1)
        dh = dh + (hv.abs() + dh) * (2.0 ** -8 + 2.0 ** -4) + 2.0 ** -10 / 224 * 1.1 * top
        wd = weights64(ew.wdtype, ew.down[e or 0], None if ew.s_down is None else ew.s_down[e or 0])
        yv = hv @ wd.T
        dy = dh @ wd.abs().T + I * 2.0 ** -23 * ((hv.abs() + dh) @ wd.abs().T)
        ref[t] += g * yv
        tol[t] += g * (dy + 2.0 ** -8 * (yv.abs() + dy))
    err = (out.cpu().view(torch.bfloat16).double() - ref).abs()
    assert bool((err <= 1.001 * tol + 2.0 ** -8 * (ref.abs() + tol)).all())


@pytest.mark.parametrize("T,act", [(3, "bf16"), (40, "bf16"), (40, "fp8"), (300, "fp8")])
def test_graph_replays_match_eager(T, act):
    layer, inp = make(T, 512, 256, 8, 4, "fp8", seed=T)
    B = block(layer, inp, act=act)
    hidden, residual = inp["hidden"].clone(), inp["residual"].clone()
    B.capture(hidden, residual)
    for rep in range(4):
        hidden.copy_(torch.roll(inp["hidden"], rep, 0))
        residual.copy_(torch.roll(inp["residual"], 2 * rep, 0))
        got = [v.clone() for v in B.replay()]
        other = block(layer, inp, act=act)
        want = other.forward(hidden, residual)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), rep


def test_no_residual_other_stream_and_no_tokens():
    layer, inp = make(4, 512, 256, 8, 2, "fp8", seed=3)
    B = block(layer, inp)
    want = B.forward(inp["hidden"])[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, s = block(layer, inp).forward(inp["hidden"], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and s is inp["hidden"]
    none = dataclasses.replace(layer, T=0)
    out, s = block(none, inp).forward(inp["hidden"][:0], inp["residual"][:0])
    assert out.shape == s.shape == (0, 512)


@pytest.mark.parametrize("T", [1, 6, 50, 2100])
def test_a_projection_before_the_block(T):
    """Norm, FP8 projection of its codes, then the block on its output and the residual stream: the projection
    against its product in 64 bits, and the block's own stages on top."""
    H = 640
    layer, inp = make(T, H, 256, 16, 2, "fp8", seed=T + 1)
    gen = rng(T)
    w = torch.randint(0, 126, (H, H), generator=gen, dtype=torch.uint8)  # positive and below NaN ...
    w |= torch.randint(0, 2, (H, H), generator=gen, dtype=torch.uint8) << 7  # ... or negative
    s_w = torch.rand((H // 128, H // 128), generator=gen) * 2.0 ** -9
    _, _, codes, exps = moe.moe_rmsnorm_quantize_act(inp["hidden"], inp["norm_w"], normed=False)
    p = moe.moe_linear_a8(codes, exps, w.to(DEV), s_w.to(DEV))
    x = e4m3(codes) * torch.exp2(exps[:, :H // 128].cpu().double()).repeat_interleave(128, 1)
    wd = e4m3(w) * s_w.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    ref = x @ wd.T
    tol = 2 * H * 2.0 ** -23 * (x.abs() @ wd.abs().T)
    got = f64(p)
    assert bool(((got - ref).abs() <= 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * tol).all())
    B = block(layer, inp)
    out, s = B.forward(p, inp["hidden"])
    torch.cuda.synchronize()
    check_front(B, dict(inp, hidden=p, residual=inp["hidden"]), s)
    assert bool(torch.isfinite(out.view(torch.bfloat16).float()).all())


def test_layer_in_two_launches():
    layer, _ = make(6, 512, 256, 16, 3, "mxfp4", seed=2)
    L = moe.MoeLayer(6, 512, 256, 16, 3, layer.experts, layer.shared, few=True)
    want, ids, wts = moe.moe_layer_few(layer.scores, layer.x, 3, moe.expert_weights(layer.experts),
                                       moe.expert_weights(layer.shared))
    want = want.clone()
    assert torch.equal(L.forward(layer.scores, layer.x), want)
    assert torch.equal(L.topk_ids, ids) and torch.equal(L.topk_w, wts)
    L.capture(layer.scores, layer.x)
    for _ in range(3):
        L.out.zero_()
        assert torch.equal(L.replay(), want)
    with pytest.raises(ValueError):
        L.forward(layer.scores, layer.x, gate_up_events=(None, None))


def test_refusals():
    layer, _ = make(9, 512, 256, 16, 3, "fp8", seed=2)
    with pytest.raises(moe.MoeError):
        moe.MoeLayer(9, 512, 256, 16, 3, layer.experts, layer.shared, few=True)
    with pytest.raises(ValueError):
        moe.MoeLayer(4, 512, 256, 16, 3, layer.experts, layer.shared, act="fp8", few=True)
