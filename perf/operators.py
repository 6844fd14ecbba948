"""Measured cases of the transformer block's serving operators around the MoE layer.

Four operators: the RMS norm with the residual's addition and an FP8 output ("norm"), the router's
product ("router"), the whole MoE layer for a few tokens ("layer") and the FP8 product with a scale per
128-block ("linear").  With own = False `run` computes them in elementary torch operations; with own = True
it calls the library.
"""
import math
import types

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BLOCK = 128


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through the norm before an MoE layer: residual, bf16 and FP8 outputs
        dict(name="norm 1 x 7168", op="norm", rows=1, K=7168, residual=True, normed=True, quantized=True),
        # a ragged prompt, the norm of a sub-layer without a residual, FP8 output alone
        dict(name="norm 777 x 2048 fp8 only", op="norm", rows=777, K=2048, residual=False, normed=False,
             quantized=True),
        # the long prefill batch
        dict(name="norm 32768 x 7168", op="norm", rows=32768, K=7168, residual=True, normed=True, quantized=True),
        # one decoded token: 256 experts, bf16 router weights
        dict(name="router 1 x 7168 x 256", op="router", T=1, H=7168, E=256, w="bf16"),
        # a ragged prompt with a router kept in fp32, 384 experts
        dict(name="router 333 x 7168 x 384 f32", op="router", T=333, H=7168, E=384, w="f32"),
        # the long prefill batch
        dict(name="router 32768 x 7168 x 256", op="router", T=32768, H=7168, E=256, w="bf16"),
        # the smallest layer, where the launches are the cost
        dict(name="layer tiny 4 bf16", op="layer", T=4, H=256, I=128, E=16, k=2, w="bf16", score_fn="softmax",
             renorm=1, shared=True),
        # one decoded token of a 256-expert layer, FP8 weights
        dict(name="layer 1 fp8", op="layer", T=1, H=7168, I=2048, E=256, k=8, w="fp8", score_fn="sigmoid",
             renorm=1, shared=True),
        # eight decoded tokens of it, 4-bit weights
        dict(name="layer 8 mxfp4", op="layer", T=8, H=7168, I=2048, E=256, k=8, w="mxfp4", score_fn="sigmoid",
             renorm=1, shared=True),
        # one token through a projection
        dict(name="linear 1 x 2048 x 7168", op="linear", M=1, N=2048, K=7168),
        # a ragged batch through a projection whose outputs are no multiple of a tile
        dict(name="linear 200 x 1000 x 7168", op="linear", M=200, N=1000, K=7168),
        # a prefill batch
        dict(name="linear 4096 x 7168 x 7168", op="linear", M=4096, N=7168, K=7168),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "router", "layer", "linear"))
    if op == "norm":
        normed = rng.random() < 0.7
        return dict(op=op, rows=_log(rng, 1, 32768), K=128 * rng.randint(2, 56), residual=rng.random() < 0.7,
                    normed=normed, quantized=not normed or rng.random() < 0.7)
    if op == "router":
        return dict(op=op, T=_log(rng, 1, 32768), H=8 * rng.randint(32, 896), E=rng.randint(8, 384),
                    w=rng.choice(("bf16", "f32")))
    if op == "layer":
        E = _log(rng, 8, 256)
        return dict(op=op, T=rng.randint(1, 8), H=128 * rng.randint(2, 56), I=128 * rng.randint(1, 16), E=E,
                    k=rng.randint(1, 8), w=rng.choice(("fp8", "bf16", "mxfp4")),
                    score_fn=rng.choice(("sigmoid", "softmax")), renorm=rng.randint(0, 1),
                    shared=rng.random() < 0.7)
    return dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 64, 7168), K=128 * rng.randint(2, 56))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 1)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _bits(t):
    """bf16 values as the 16-bit patterns that the library's calls take."""
    return t.to(torch.bfloat16).view(torch.int16)


def _fp8(w):
    return w.to(torch.float8_e4m3fn).view(torch.uint8)


def _weights(g, kind, n, rows, cols):
    """n matrices [rows, cols] of about N(0, 0.02^2) in the weight format `kind`, with their scales."""
    if kind == "bf16":
        return _bits(_randn(g, n, rows, cols).mul_(0.02)), None
    if kind == "fp8":  # codes of N(0, 100^2), one fp32 scale per 128 x 128 block around 0.0002
        codes = torch.empty((n, rows, cols), dtype=torch.uint8, device=DEV)
        for i in range(0, n, 16):
            codes[i:i + 16] = _fp8(_randn(g, min(16, n - i), rows, cols).mul_(100.0).clamp_(-448.0, 448.0))
        s = torch.rand((n, -(-rows // BLOCK), cols // BLOCK), generator=g, device=DEV).mul_(1e-4).add_(1.5e-4)
        return codes, s
    codes = torch.randint(0, 256, (n, rows, cols // 2), generator=g, device=DEV, dtype=torch.uint8)
    # E2M1 codes uniform (root mean square 2.9) with E8M0 scales 2^-8, 2^-7 and 2^-6
    return codes, torch.randint(119, 122, (n, rows, cols // 32), generator=g, device=DEV, dtype=torch.uint8)


def _experts(g, c, n):
    gate, s_gate = _weights(g, c["w"], n, c["I"], c["H"])
    up, s_up = _weights(g, c["w"], n, c["I"], c["H"])
    down, s_down = _weights(g, c["w"], n, c["H"], c["I"])
    return types.SimpleNamespace(wdtype=c["w"], gate=gate, up=up, down=down, s_gate=s_gate, s_up=s_up,
                                 s_down=s_down)


def prepare(case, seed):
    g = _gen(seed)
    st = types.SimpleNamespace(**case)
    if case["op"] == "norm":
        # a residual stream grows with depth, a sub-layer's output is smaller; a few large channels
        loud = 1.0 + 15.0 * (torch.rand((case["K"],), generator=g, device=DEV) < 0.005)
        st.x = _bits(_randn(g, case["rows"], case["K"]) * loud)
        st.res = _bits(_randn(g, case["rows"], case["K"]) * (4.0 * loud)) if case["residual"] else None
        st.g = _bits(1.0 + 0.1 * _randn(g, case["K"]))
    elif case["op"] == "router":
        st.x = _bits(_randn(g, case["T"], case["H"]))
        w = _randn(g, case["E"], case["H"]).mul_(0.02)
        st.wr = w if case["w"] == "f32" else _bits(w)
    elif case["op"] == "layer":
        st.x = _bits(_randn(g, case["T"], case["H"]))
        st.scores = _randn(g, case["T"], case["E"])
        st.experts = _experts(g, case, case["E"])
        st.sh = _experts(g, case, 1) if case["shared"] else None
    else:
        st.codes = _fp8(_randn(g, case["M"], case["K"]).mul_(100.0).clamp_(-448.0, 448.0))
        st.exps = torch.randint(-8, -3, (case["M"], -(-case["K"] // 2048) * 16), generator=g, device=DEV,
                                dtype=torch.int8)
        w, s = _weights(g, "fp8", 1, case["N"], case["K"])
        st.wl, st.sl = w[0], s[0]
    if own:  # what a user's program keeps: weight handles, workspace and output buffers
        import routed_expert_grouped_amd as moe
        st.moe = moe
        e = lambda shape, t: torch.empty(shape, dtype=t, device=DEV)  # noqa: E731
        if case["op"] == "norm":
            shape = (case["rows"], case["K"])
            st.sum_ = e(shape, torch.int16) if case["residual"] else None
            st.y = e(shape, torch.int16) if case["normed"] else None
            st.q = e(shape, torch.uint8) if case["quantized"] else None
            st.qe = e((case["rows"], moe.exp_pitch(case["K"])), torch.int8) if case["quantized"] else None
        elif case["op"] == "router":
            st.out = e((case["T"], case["E"]), torch.float32)
        elif case["op"] == "layer":
            st.w_ = moe.expert_weights(st.experts)
            st.ws_ = moe.expert_weights(st.sh) if st.sh is not None else None
            st.ids = e((case["T"], case["k"]), torch.int32)
            st.tw = e((case["T"], case["k"]), torch.float32)
            st.out = e((case["T"], case["H"]), torch.int16)
            st.work = e((max(16, moe.moe_layer_few_workspace_size(case["T"], case["k"], st.w_)),), torch.uint8)
        else:
            st.out = e((case["M"], case["N"]), torch.int16)
    return st


# ---------------------------------------------------------------- plain forms

def _f(bits):
    return bits.view(torch.bfloat16).float()


def _pow2(e):
    """2^e for whole numbers e of a normal float's range, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _dequant(kind, w, s):
    """Weights [..., rows, cols] as fp32."""
    if kind == "bf16":
        return _f(w)
    if kind == "mxfp4":
        lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
        lut = torch.cat([lut, -lut])
        v = torch.stack([lut[(w & 15).int()], lut[(w >> 4).int()]], -1).flatten(-2)
        return (v.unflatten(-1, (-1, 32)) * _pow2(s.int() - 127)[..., None]).flatten(-2)
    v = w.view(torch.float8_e4m3fn).float()
    sc = s.repeat_interleave(BLOCK, -2)[..., :v.shape[-2], :]  # a scale per row and 128 columns
    return (v.unflatten(-1, (-1, BLOCK)) * sc[..., None]).flatten(-2)


def _plain_norm(st):
    v = _f(st.x)
    if st.residual:
        v = (v + _f(st.res)).to(torch.bfloat16)
    total = v if st.residual else None
    # 64 bits up to one rounding to fp32: the 8-bit rounding has values next to its borders
    d = v.double()
    r = 1.0 / torch.sqrt(d.square().mean(-1, keepdim=True) + EPS)
    y = (d * r * _f(st.g).double()).float()
    codes = exps = None
    if st.quantized:
        blk = y.unflatten(-1, (-1, BLOCK))
        amax = blk.abs().amax(-1)
        m, e2 = torch.frexp(amax)
        e = torch.where(m <= 0.875, e2 - 9, e2 - 8)
        e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp(-126, 126)
        codes = (blk * _pow2(-e)[..., None]).flatten(-2).to(torch.float8_e4m3fn)
        exps = e.to(torch.int8)
    return dict(total=total, y=y.to(torch.bfloat16) if st.normed else None, codes=codes, exps=exps)


def _plain_layer(st):
    T, k = st.T, st.k
    s = st.scores.double()
    ids = torch.sort(st.scores, dim=-1, descending=True, stable=True).indices[:, :k]
    top = s.gather(-1, ids)
    if st.score_fn == "softmax":
        num = torch.exp(top - top[:, :1])
        den = num.sum(-1, keepdim=True) if st.renorm else torch.exp(s - top[:, :1]).sum(-1, keepdim=True)
    else:
        num = 1.0 / (1.0 + torch.exp(-top))
        den = num.sum(-1, keepdim=True) if st.renorm else torch.ones_like(num)
    tw = (num / den).float()
    x = _f(st.x)

    def ffn(w, pick, xs):
        part = lambda t: None if t is None else t[pick]  # noqa: E731
        a = torch.matmul(_dequant(st.w, part(w.gate), part(w.s_gate)), xs)
        b = torch.matmul(_dequant(st.w, part(w.up), part(w.s_up)), xs)
        h = a / (1.0 + torch.exp(-a)) * b
        return torch.matmul(_dequant(st.w, part(w.down), part(w.s_down)), h)

    flat = ids.reshape(-1)
    y = ffn(st.experts, flat, x.repeat_interleave(k, 0)[:, :, None]).reshape(T, k, -1)
    out = (y * tw[:, :, None]).sum(1)
    if st.sh is not None:
        out = out + ffn(st.sh, slice(0, 1), x.T[None])[0].T
    return dict(out=out.to(torch.bfloat16), ids=ids.to(torch.int32), w=tw)


def _plain(st):
    if st.op == "norm":
        return _plain_norm(st)
    if st.op == "router":
        return dict(scores=_f(st.x) @ (st.wr if st.w == "f32" else _f(st.wr)).T)
    if st.op == "layer":
        return _plain_layer(st)
    kb = st.K // BLOCK
    x = (st.codes.view(torch.float8_e4m3fn).float().unflatten(-1, (kb, BLOCK))
         * _pow2(st.exps[:, :kb])[..., None]).flatten(-2)
    return dict(out=(x @ _dequant("fp8", st.wl, st.sl).T).to(torch.bfloat16))


def run(st):
    if not own:
        return _plain(st)
    moe = st.moe
    b16 = lambda t: None if t is None else t.view(torch.bfloat16)  # noqa: E731
    if st.op == "norm":
        total, y, codes, exps = moe.moe_rmsnorm_quantize_act(
            st.x, st.g, residual=st.res, eps=EPS, normed=st.normed, quantized=st.quantized, sum_out=st.sum_,
            y=st.y, codes=st.q, exps=st.qe)
        return dict(total=b16(total), y=b16(y),
                    codes=None if codes is None else codes.view(torch.float8_e4m3fn),
                    exps=None if exps is None else exps[:, :st.K // BLOCK])
    if st.op == "router":
        return dict(scores=moe.moe_router_scores(st.x, st.wr, scores=st.out))
    if st.op == "layer":
        out, ids, tw = moe.moe_layer_few(st.scores, st.x, st.k, st.w_, st.ws_, score_fn=st.score_fn,
                                         renorm=st.renorm, topk_ids=st.ids, topk_w=st.tw, out=st.out,
                                         work=st.work)
        return dict(out=b16(out), ids=ids, w=tw)
    return dict(out=b16(moe.moe_linear_a8(st.codes, st.exps, st.wl, st.sl, y=st.out)))


# ---------------------------------------------------------------- work

def work(case):
    c = types.SimpleNamespace(**case)
    if c.op == "norm":
        n = c.rows * c.K
        per = 2 + (4 if c.residual else 0) + (2 if c.normed else 0) + (1 + 1 / BLOCK if c.quantized else 0)
        return {"bytes": n * per + 2 * c.K, "flops": 6 * n}
    if c.op == "router":
        return {"bytes": 2 * c.T * c.H + (4 if c.w == "f32" else 2) * c.E * c.H + 4 * c.T * c.E,
                "flops": 2 * c.T * c.H * c.E}
    if c.op == "layer":
        touched = c.E * (1.0 - (1.0 - c.k / c.E) ** c.T) + (1 if c.shared else 0)  # expected, distinct
        per = {"bf16": 2.0, "fp8": 1.0 + 4.0 / BLOCK ** 2, "mxfp4": 0.5 + 1.0 / 32}[c.w]
        return {"bytes": touched * 3 * c.H * c.I * per + c.T * (4 * c.H + 4 * c.E + 8 * c.k),
                "flops": 6 * c.H * c.I * c.T * (c.k + (1 if c.shared else 0))}
    kb = c.K // BLOCK
    return {"bytes": c.M * (c.K + kb) + c.N * c.K + 4 * -(-c.N // BLOCK) * kb + 2 * c.M * c.N,
            "flops": 2 * c.M * c.N * c.K}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _values64(kind, w, s):
    """One matrix [rows, cols] in 64 bits, from the formats' definitions."""
    if kind == "bf16":
        return w.view(torch.bfloat16).to(torch.float64)
    if kind == "fp8":  # sign, 4 exponent bits (bias 7), 3 mantissa bits
        c = w.to(torch.int64)
        ex, man = (c >> 3) & 15, (c & 7).double()
        mag = torch.where(ex > 0, (1 + man / 8) * torch.pow(2.0, (ex - 7).double()), man * 2.0 ** -9)
        v = torch.where(c >= 128, -mag, mag)
        rows = torch.arange(w.shape[0], device=w.device) // BLOCK
        cols = torch.arange(w.shape[1], device=w.device) // BLOCK
        return v * s.double()[rows][:, cols]
    lo, hi = w.to(torch.int64) & 15, w.to(torch.int64) >> 4
    c = torch.empty((w.shape[0], 2 * w.shape[1]), dtype=torch.int64, device=w.device)
    c[:, 0::2], c[:, 1::2] = lo, hi
    ex, man = (c >> 1) & 3, (c & 1).double()  # sign, 2 exponent bits (bias 1), 1 mantissa bit
    mag = torch.where(ex > 0, (1 + man / 2) * torch.pow(2.0, (ex - 1).double()), man * 0.5)
    cols = torch.arange(c.shape[1], device=w.device) // 32
    return torch.where(c >= 8, -mag, mag) * torch.pow(2.0, s.double() - 127)[:, cols]


def exact(case, seed):
    st = prepare(case, seed)
    if st.op == "norm":
        def norm_rows(lo, hi):
            v = st.x[lo:hi].view(torch.bfloat16).double()
            total = None
            if st.residual:
                total = v + st.res[lo:hi].view(torch.bfloat16).double()
                v = total.to(torch.bfloat16).double()  # what is normalised is the stored sum
            y = v * st.g.view(torch.bfloat16).double() * (v.pow(2).sum(-1, keepdim=True) / st.K + EPS).pow(-0.5)
            codes = exps = None
            if st.quantized:
                blocks = y.reshape(hi - lo, -1, BLOCK)
                ratio = blocks.abs().max(-1).values / 448
                exps = torch.where(ratio > 0, torch.ceil(torch.log2(ratio)), 0.0)
                codes = (blocks / torch.pow(2.0, exps)[..., None]).reshape(hi - lo, -1)
            return total, y if st.normed else None, codes, exps
        parts = [norm_rows(i, min(st.rows, i + 8192)) for i in range(0, st.rows, 8192)]
        cat = [None if p[0] is None else torch.cat(p) for p in zip(*parts)]
        return dict(total=cat[0], y=cat[1], codes=cat[2],
                    exps=None if cat[3] is None else cat[3].to(torch.int8))
    if st.op == "router":
        w = st.wr.double() if st.w == "f32" else st.wr.view(torch.bfloat16).double()
        return dict(scores=torch.mm(st.x.view(torch.bfloat16).double(), w.t()))
    if st.op == "linear":
        a = _values64("fp8", st.codes, torch.ones((-(-st.M // BLOCK), st.K // BLOCK), device=DEV))
        per = torch.pow(2.0, st.exps.double())
        for b in range(st.K // BLOCK):
            a[:, b * BLOCK:(b + 1) * BLOCK] *= per[:, b:b + 1]
        return dict(out=torch.mm(a, _values64("fp8", st.wl, st.sl).t()))
    ids, tw = [], []
    for row in st.scores.cpu().tolist():
        order = sorted(range(st.E), key=lambda e: (-row[e], e))[:st.k]
        if st.score_fn == "softmax":
            num = [math.exp(row[e] - row[order[0]]) for e in order]
            den = math.fsum(num) if st.renorm else math.fsum(math.exp(v - row[order[0]]) for v in row)
        else:
            num = [1 / (1 + math.exp(-row[e])) for e in order]
            den = math.fsum(num) if st.renorm else 1.0
        ids.append(order)
        tw.append([n / den for n in num])
    x = st.x.view(torch.bfloat16).double()
    out = torch.zeros((st.T, st.H), dtype=torch.float64, device=DEV)

    def expert(w, e, xt):
        sc = lambda t: None if t is None else t[e]  # noqa: E731
        a = torch.mm(xt, _values64(st.w, w.gate[e], sc(w.s_gate)).t())
        b = torch.mm(xt, _values64(st.w, w.up[e], sc(w.s_up)).t())
        return torch.mm(a * torch.sigmoid(a) * b, _values64(st.w, w.down[e], sc(w.s_down)).t())

    for e in sorted({e for row in ids for e in row}):
        who = [(t, tw[t][row.index(e)]) for t, row in enumerate(ids) if e in row]
        at = torch.tensor([t for t, _ in who], device=DEV)
        gate = torch.tensor([g for _, g in who], dtype=torch.float64, device=DEV)
        out[at] += gate[:, None] * expert(st.experts, e, x[at])
    if st.sh is not None:
        out += expert(st.sh, 0, x)
    return dict(out=out, ids=torch.tensor(ids, dtype=torch.int32, device=DEV),
                w=torch.tensor(tw, dtype=torch.float64, device=DEV))
