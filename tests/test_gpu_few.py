"""moe_layer_few against the layer's formula in 64 bits (block_util.layer64 derives the tolerance), its
routing against moe_route bit for bit, and what a token's output may depend on."""
import dataclasses

import pytest
import torch

import routed_expert_grouped_amd as moe
import synth
from block_util import DEV, Guarded, layer64

pytestmark = pytest.mark.gpu


def make(T, H, I, E, k, wdtype, seed=0, score_fn="sigmoid", renorm=1, shared=True):
    big = H * I * E > 1 << 26
    cfg = dict(T=T, H=H, I=I, E=E, k=k, score_fn=score_fn, renorm=renorm, scores="normal", wdtype=wdtype)
    layer = synth.make_layer(cfg, seed=seed, device=DEV) if big else synth.make_layer(cfg, seed=seed).to(DEV)
    return layer if shared else dataclasses.replace(layer, shared=None)


def run(layer, guard=True, **kw):
    T, k = layer.T, layer.k
    w = moe.expert_weights(layer.experts)
    ws = moe.expert_weights(layer.shared) if layer.shared is not None else None
    G = Guarded()
    got = moe.moe_layer_few(layer.scores, layer.x, k, w, ws, layer.score_fn, layer.renorm,
                            topk_ids=G((T, k), torch.int32), topk_w=G((T, k), torch.float32),
                            out=G((T, layer.H), torch.int16),
                            work=G((moe.moe_layer_few_workspace_size(T, k, w),), torch.uint8), **kw)
    G.check()
    return got


def check(layer):
    out, ids, wts = run(layer)
    want_ids, want_w = moe.moe_route(layer.scores, layer.k, layer.score_fn, layer.renorm)
    torch.cuda.synchronize()
    assert torch.equal(ids, want_ids) and torch.equal(wts, want_w)
    ref, tol = layer64(layer, ids.cpu(), wts.cpu())
    got = out.view(torch.bfloat16).double()
    assert bool(((got - ref).abs() <= ref.abs() * 2.0 ** -8 + (1 + 2.0 ** -8) * tol).all())
    # bf16's half step bounds a row's relative error by 2^-8; the rest is some 2^-15
    rel = (got - ref).norm(dim=1) / ref.norm(dim=1)
    assert float(rel.max()) <= 2.0 ** -8 + 2.0 ** -11, float(rel.max())
    return out


SHAPES = [  # T, H, I, E, k
    (1, 128, 128, 1, 1),        # one expert, one block: seven of eight waves have no stage
    (1, 256, 128, 16, 2), (4, 256, 128, 16, 2), (8, 256, 128, 16, 2),
    (2, 384, 256, 8, 8),        # every expert, odd blocks
    (3, 640, 384, 65, 3),       # 128 scores a row and a few
    (5, 1152, 640, 130, 4),     # nine blocks a row, five down
    (6, 512, 896, 300, 5),
    (7, 896, 256, 600, 6),
    (8, 256, 128, 1024, 32),    # the most experts and slots: 256 assignments
    (8, 1024, 128, 64, 1),
    (3, 128, 4224, 4, 2),       # more units of one expert than workgroups
    (8, 7168, 256, 32, 8),      # the longest x that eight tokens may have
    (2, 16384, 128, 4, 2),
    (3, 16384, 384, 6, 3),
    (1, 2048, 7168, 3, 2),
    # several workgroups a tile of the down phase (and shares of them without a stage)
    (8, 1024, 512, 40, 8), (4, 2048, 1408, 16, 6), (8, 4096, 640, 24, 6), (8, 5120, 512, 30, 8),
    (2, 2048, 1408, 8, 8), (8, 256, 2048, 48, 8),
]


@pytest.mark.parametrize("wdtype", ["fp8", "bf16", "mxfp4"])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, wdtype):
    check(make(*shape, wdtype, seed=sum(shape)))


@pytest.mark.parametrize("wdtype", ["fp8", "bf16", "mxfp4"])
@pytest.mark.parametrize("score_fn,renorm,shared", [("softmax", 1, True), ("softmax", 0, False),
                                                    ("sigmoid", 0, True), ("sigmoid", 1, False)])
def test_routing_rules_and_no_shared_expert(wdtype, score_fn, renorm, shared):
    for T, I in ((1, 128), (3, 4224), (8, 384)):
        check(make(T, 256, I, 20, 3, wdtype, seed=T, score_fn=score_fn, renorm=renorm, shared=shared))


@pytest.mark.parametrize("wdtype", ["fp8", "bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 8])
def test_full_size(wdtype, T):
    if wdtype == "bf16":
        layer = make(T, 7168, 2048, 24, 8, wdtype, seed=3)
    else:
        layer = make(T, 7168, 2048, 64, 8, wdtype, seed=3)
    check(layer)


@pytest.mark.parametrize("wdtype", ["fp8", "bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 5])
def test_rows_of_a_wide_range(wdtype, T):
    """Values from 2^-40 to 2^40 in one block, blocks of zeros, the smallest values of the type, and a sum that
    only the small ones make."""
    layer = make(T, 512, 256, 12, 3, wdtype, seed=40 + T)
    gen = torch.Generator().manual_seed(T)
    v = layer.x.cpu().view(torch.bfloat16).float()
    v *= torch.exp2(torch.randint(-40, 41, v.shape, generator=gen).float())
    v[:, 128:256] = 0.0
    v[:, 256:384] = torch.randint(-3, 4, (T, 128), generator=gen) * 2.0 ** -133
    v[0] = 0.0
    v[0, 384:] = layer.x[0, 384:].cpu().view(torch.bfloat16).float() * 2.0 ** -100
    layer.x.copy_(v.to(torch.bfloat16).view(torch.int16))
    out, ids, wts = run(layer)
    ref, tol = layer64(layer, ids.cpu(), wts.cpu())
    assert bool(((out.view(torch.bfloat16).double() - ref).abs() <= ref.abs() * 2.0 ** -8 + (1 + 2.0 ** -8) * tol + 2.0 ** -126).all())


def test_all_tokens_on_one_expert():
    layer = make(8, 512, 256, 12, 1, "fp8", seed=4)
    layer.scores.fill_(0.0)
    layer.scores[:, 7] = 1.0
    out = check(layer)
    same = dataclasses.replace(layer, x=layer.x[:1].expand(8, -1).contiguous())
    out = run(same)[0]
    assert bool((out == out[:1]).all())


def test_ties_go_to_the_lower_expert():
    layer = make(4, 256, 128, 70, 6, "fp8", seed=5)
    layer.scores.copy_(torch.randint(0, 3, layer.scores.shape, generator=torch.Generator().manual_seed(1)).float())
    check(layer)


@pytest.mark.parametrize("wdtype", ["fp8", "bf16", "mxfp4"])
def test_a_token_depends_on_its_own_row_and_experts(wdtype):
    """Experts that a token is not routed to may hold anything (NaN codes, NaN scales, infinities), and so
    may other tokens' rows; experts that no token is routed to are not read."""
    layer = make(6, 512, 384, 16, 2, wdtype, seed=6)
    out, ids, _ = run(layer)
    ids = ids.cpu()
    bad = int(ids[0, 0])
    clean = [t for t in range(6) if bad not in ids[t].tolist()]
    untouched = [e for e in range(16) if e not in ids.flatten().tolist()]
    assert clean and untouched
    ew = layer.experts
    for e in [bad] + untouched:
        if wdtype == "bf16":
            ew.gate[e], ew.up[e], ew.down[e] = 0x7FC0, 0x7F80, 0x7FC0
        elif wdtype == "fp8":
            ew.gate[e], ew.down[e], ew.s_up[e] = 0x7F, 0xFF, float("inf")
        else:
            ew.s_gate[e], ew.s_down[e] = 255, 255
    got = run(layer)[0]
    assert torch.equal(got[clean], out[clean])
    assert bool(torch.isnan(got[0].view(torch.bfloat16).float()).all())
    layer2 = make(6, 512, 384, 16, 2, wdtype, seed=6)
    layer2.x[3, 17] = 0x7FC0
    layer2.x[1, 40] = 0x7F80
    got = run(layer2)[0]
    keep = [0, 2, 4, 5]
    assert torch.equal(got[keep], out[keep])
    assert bool(torch.isnan(got[3].view(torch.bfloat16).float()).all())


def test_zero_scales_and_zero_rows():
    layer = make(4, 512, 256, 8, 2, "fp8", seed=7)
    layer.experts.s_gate[:, 0, 1] = 0.0
    layer.experts.s_down[:, 2, 0] = 0.0
    layer.shared.s_up[:] = 0.0
    layer.x[2] = 0
    out = check_rows(layer, [0, 1, 3])
    assert bool((out[2] == 0).all())


def check_rows(layer, rows):
    out, ids, wts = run(layer)
    ref, tol = layer64(layer, ids.cpu(), wts.cpu())
    got = out.view(torch.bfloat16).double()
    assert bool(((got - ref).abs() <= ref.abs() * 2.0 ** -8 + (1 + 2.0 ** -8) * tol)[rows].all())
    return out


def test_equal_inputs_give_equal_bits_and_nothing_is_kept():
    """Calls of other sizes in between, and a workspace full of NaN patterns, change nothing."""
    a, b = make(5, 640, 384, 40, 4, "fp8", seed=8), make(2, 256, 128, 16, 2, "mxfp4", seed=9)
    w = moe.expert_weights(a.experts)
    ws = moe.expert_weights(a.shared)
    work = torch.full((moe.moe_layer_few_workspace_size(5, 4, w),), 255, dtype=torch.uint8, device=DEV)
    first = run(a)[0].clone()
    run(b)
    got = moe.moe_layer_few(a.scores, a.x, 4, w, ws, work=work)[0]
    assert torch.equal(got, first)
    assert torch.equal(moe.moe_layer_few(a.scores, a.x, 4, w, ws)[0], first)


def test_close_to_the_separate_calls():
    """MoeLayer rounds h and y to bf16 on the way: the two agree to a few bf16 half steps a row."""
    layer = make(8, 1024, 512, 32, 4, "fp8", seed=10)
    L = moe.MoeLayer(8, 1024, 512, 32, 4, layer.experts, layer.shared, "sigmoid", 1)
    a = L.forward(layer.scores, layer.x).view(torch.bfloat16).double()
    b = run(layer)[0].view(torch.bfloat16).double()
    assert float(((a - b).norm(dim=1) / b.norm(dim=1)).max()) <= 1e-2


@pytest.mark.parametrize("wdtype", ["fp8", "mxfp4"])
def test_streams_and_graph(wdtype):
    layer = make(4, 512, 256, 24, 3, wdtype, seed=11)
    scores, x = layer.scores.clone(), layer.x.clone()
    w, ws = moe.expert_weights(layer.experts), moe.expert_weights(layer.shared)
    call = lambda **kw: moe.moe_layer_few(scores, x, 3, w, ws, **kw)  # noqa: E731
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    bufs = dict(out=torch.zeros_like(want[0]), topk_ids=torch.zeros_like(want[1]), topk_w=torch.zeros_like(want[2]),
                work=torch.empty(moe.moe_layer_few_workspace_size(4, 3, w), dtype=torch.uint8, device=DEV))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(**bufs)
    for rep in range(5):
        if rep >= 3:
            scores.copy_(torch.roll(scores, 1, 0))
            x.copy_(torch.roll(x, 2, 0))
            want = [t.clone() for t in call()]
        bufs["work"].fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((bufs["out"], bufs["topk_ids"], bufs["topk_w"]), want))


def test_two_calls_at_once():
    """Two calls on two streams, each with its own workspace."""
    a, b = make(8, 1024, 512, 32, 4, "fp8", seed=12), make(3, 2048, 384, 16, 2, "fp8", seed=13)
    want = [run(a)[0].clone(), run(b)[0].clone()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for layer, s in zip((a, b), streams):
            outs.append(moe.moe_layer_few(layer.scores, layer.x, layer.k, moe.expert_weights(layer.experts),
                                          moe.expert_weights(layer.shared), stream=s)[0])
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2])


def test_no_tokens_and_refusals():
    layer = make(4, 256, 128, 16, 2, "fp8", seed=14)
    w, ws = moe.expert_weights(layer.experts), moe.expert_weights(layer.shared)
    out, ids, wts = moe.moe_layer_few(layer.scores[:0], layer.x[:0], 2, w, ws)
    assert out.shape == (0, 256) and ids.shape == (0, 2)
    for kw in (dict(scores=layer.scores[:, :8]), dict(scores=layer.scores.double()), dict(x=layer.x[:2]),
               dict(x=layer.x.t()), dict(x=layer.x.cpu()), dict(out=torch.empty((4, 255), device=DEV)),
               dict(topk_ids=torch.empty((4, 2), dtype=torch.int64, device=DEV))):
        with pytest.raises(ValueError):
            moe.moe_layer_few(**(dict(scores=layer.scores, x=layer.x, k=2, w=w, shared=ws) | kw))
    nine = torch.zeros((9, 16), device=DEV), torch.zeros((9, 256), dtype=torch.int16, device=DEV)
    with pytest.raises(moe.MoeError) as e:
        moe.moe_layer_few(*nine, 2, w, ws)
    assert e.value.status == moe.MOE_ERR_UNSUPPORTED
    with pytest.raises(moe.MoeError) as e:
        moe.moe_layer_few(layer.scores, layer.x, 2, w, ws, work=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == moe.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("wdtype", ["fp8", "bf16", "mxfp4"])
def test_shared_tiles_give_equal_bits_every_time(wdtype):
    """Several workgroups add to a tile of the down phase, in an order that must not show: eager, with any
    workspace contents, on two streams at once, and replayed."""
    layer = make(8, 1024, 512, 40, 8, wdtype, seed=12)
    w, ws = moe.expert_weights(layer.experts), moe.expert_weights(layer.shared)
    works = [torch.empty(moe.moe_layer_few_workspace_size(8, 8, w), dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [torch.empty((8, 1024), dtype=torch.int16, device=DEV) for _ in range(2)]
    want = run(layer)[0].clone()

    def call(i, **kw):
        moe.moe_layer_few(layer.scores, layer.x, 8, w, ws, layer.score_fn, layer.renorm, out=outs[i], work=works[i], **kw)
    for fill in (0, 1, 255, None, None):
        if fill is not None:
            works[0].fill_(fill)
        call(0)
        assert torch.equal(outs[0], want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            call(i, stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    for _ in range(5):
        outs[0].zero_()
        works[0].fill_(170)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want)
