"""Cases that measure four operators of the MoE layer library, each with its plain form.

  mx       MXFP4 quantisation of rows and back (moe_mx_quantize, moe_mx_dequantize)
  ffn      the grouped SwiGLU expert products on MXFP4 weights and activations (MoeLayer, wt = "mxfp4")
  layer    one forward pass of that layer, router to combine
  balance  the router's load-balance loss with per-expert counts, and its gradient (moe_balance_loss[_backward])
  norm     the norms around the layer: y = x + rs * gate * rms(block) * w_post, xn = rms(y) * w_pre, and their
           gradient (moe_block_norm[_backward])

MXFP4 here is the OCP Microscaling format: blocks of 32 along a row share one power-of-two scale (a byte, exponent
biased by 127), the elements are E2M1 codes, two to a byte, the even column in the low nibble.  A block's exponent is
floor(log2(largest magnitude)) - 2, kept within [-127, 125]; an all-zero block has scale 1; a block with a NaN or an
infinity has the scale byte 255 and stands for NaN.

`run` computes the plain form with elementary torch operations in 32 bits where `own` is false, and calls the
library where it is true."""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch's hidden states on the way to FP4 experts
        {"name": "mx_decode_rows", "kind": "mx", "rows": 128, "cols": 7168, "dtype": "bf16"},
        # one Mixtral-shaped expert's gate/up weights, quantised from fp32 when a model is loaded
        {"name": "mx_expert_weights", "kind": "mx", "rows": 28672, "cols": 4096, "dtype": "f32"},
        # Mixtral-8x7B-shaped decode step: few large experts, 32 tokens
        {"name": "ffn_decode_8_experts", "kind": "ffn", "T": 32, "H": 4096, "I": 14336, "E": 8, "K": 2,
         "layout": "masked"},
        # DeepSeek-V3-shaped decode step: many experts with a handful of tokens each
        {"name": "ffn_decode_256_experts", "kind": "ffn", "T": 128, "H": 7168, "I": 2048, "E": 256, "K": 8,
         "layout": "masked"},
        # the prefill workload: 8192 tokens over 512 experts, ragged contiguous groups
        {"name": "ffn_prefill_512_experts", "kind": "ffn", "T": 8192, "H": 4096, "I": 1024, "E": 512, "K": 10,
         "layout": "contig"},
        # one dense expert over a long prompt (a shared expert, or a dense layer): bound by the tensor cores
        {"name": "ffn_prefill_dense", "kind": "ffn", "T": 8192, "H": 4096, "I": 14336, "E": 1, "K": 1,
         "layout": "contig"},
        # a single token through the whole layer, where each launch's latency counts
        {"name": "layer_one_token", "kind": "layer", "T": 1, "H": 4096, "I": 14336, "E": 8, "K": 2},
        # a small training micro-batch
        {"name": "balance_small", "kind": "balance", "T": 128, "E": 256, "K": 8, "B": 1, "score": "softmax",
         "pad": 0.0},
        # the prefill workload's router in training, the loss over the whole batch
        {"name": "balance_batch", "kind": "balance", "T": 8192, "E": 512, "K": 10, "B": 1, "score": "softmax",
         "pad": 0.0},
        # packed sequences of very different lengths with padding, sigmoid scores, one loss per sequence
        {"name": "balance_packed", "kind": "balance", "T": 65536, "E": 256, "K": 8, "B": 48, "score": "sigmoid",
         "pad": 0.1},
        # a decode step: the layer's output normed, gated and added, and the next block's input normed
        {"name": "norm_decode", "kind": "norm", "T": 128, "H": 7168, "dtype": "bf16", "gate": "channel",
         "train": False},
        # a training step's forward and backward with one gate value a token
        {"name": "norm_train", "kind": "norm", "T": 8192, "H": 4096, "dtype": "bf16", "gate": "token",
         "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    """A multiple of m, spread over the logarithm of [lo, hi]."""
    while True:
        v = max(lo, min(hi, _log(rng, lo, hi) // m * m))
        if v != 24 * 128:
            return v


def draw(rng):
    kind = rng.choice(["mx", "ffn", "ffn", "layer", "balance", "balance", "norm", "norm"])
    if kind == "mx":
        while True:
            c = {"kind": kind, "rows": _log(rng, 1, 28672), "cols": _mult(rng, 32, 14336, 32),
                 "dtype": rng.choice(["bf16", "f32"])}
            if c["rows"] * c["cols"] <= 28672 * 4096:
                return c
    if kind == "ffn":
        while True:
            E = _log(rng, 1, 512)
            c = {"kind": kind, "T": _log(rng, 1, 8192), "H": _mult(rng, 128, 7168, 128),
                 "I": _mult(rng, 128, 14336, 128), "E": E, "K": rng.randint(1, min(E, 10)),
                 "layout": rng.choice(["masked", "contig"])}
            w = c["E"] * c["H"] * c["I"]
            if w <= 256 * 7168 * 2048 and c["T"] * c["K"] * c["H"] * c["I"] <= 8192 * 10 * 4096 * 1024:
                return c
    if kind == "layer":
        while True:
            E = _log(rng, 1, 64)
            T = rng.randint(1, 8)
            c = {"kind": kind, "T": T, "H": _mult(rng, 128, 7168, 128), "I": _mult(rng, 128, 14336, 128), "E": E,
                 "K": rng.randint(1, min(E, 8, max(1, 16 // T)))}
            if c["E"] * c["H"] * c["I"] <= 8 * 4096 * 14336:
                return c
    if kind == "balance":
        while True:
            E = _log(rng, 2, 1024)
            T = _log(rng, 1, 65536)
            c = {"kind": kind, "T": T, "E": E, "K": rng.randint(1, min(E, 10)),
                 "B": _log(rng, 1, min(64, T)), "score": rng.choice(["softmax", "sigmoid"]),
                 "pad": rng.choice([0.0, 0.05, 0.2])}
            if T * E <= 65536 * 256:
                return c
    while True:
        H = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            H = H // 8 * 8
        c = {"kind": kind, "T": _log(rng, 1, 16384), "H": H, "dtype": rng.choice(["bf16", "bf16", "f32"]),
             "gate": rng.choice(["none", "channel", "token"]), "train": rng.random() < 0.6}
        if c["T"] * H <= (8192 * 4096 if c["dtype"] == "bf16" else 8192 * 2048) and H != 24 * 128:
            return c


def work(case):
    c = case
    if c["kind"] == "mx":
        n, es = c["rows"] * c["cols"], 2 if c["dtype"] == "bf16" else 4
        # the rows, the codes and scales that are kept, the values they stand for
        return {"bytes": n * es + n * 17 / 32 + n * es, "flops": 0}
    if c["kind"] in ("ffn", "layer"):
        rows, w = c["T"] * c["K"], 3 * c["H"] * c["I"]
        touched = c["E"] * (1.0 - (1.0 - c["K"] / c["E"]) ** c["T"])
        if c["kind"] == "ffn":
            act = rows * c["H"] * 17 / 32 + rows * c["H"] * 2
        else:
            act = c["T"] * (c["H"] * 2 + c["E"] * 4 + c["H"] * 2)
        return {"bytes": touched * w * 17 / 32 + act, "flops": 2.0 * rows * w}
    if c["kind"] == "balance":
        n = c["T"] * c["E"]
        # logits once for the loss and once for the gradient (which needs every token's counts first)
        return {"bytes": 12 * n + 4 * c["T"] * c["K"] + 12 * c["B"] * c["E"], "flops": 12 * n}
    n, es = c["T"] * c["H"], 2 if c["dtype"] == "bf16" else 4
    # forward: x, block -> y, xn; backward: x, block, dy, dxn -> dx, dblock
    return {"bytes": n * es * (10 if c["train"] else 4), "flops": n * (40 if c["train"] else 12)}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * std


def _weights(g, n, rows, cols):
    """n experts' weights, N(0, 0.02), as MXFP4 codes and scales."""
    codes = torch.empty(n, rows, cols // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(n, rows, cols // 32, dtype=torch.uint8, device=DEV)
    for e in range(n):
        codes[e], scales[e] = _quantise(_normal(g, rows, cols, std=0.02))
    return codes, scales


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["kind"] == "mx":
        dt = _dtype(c["dtype"])
        s["x"] = _normal(g, c["rows"], c["cols"], std=1.0 if c["dtype"] == "bf16" else 0.02).to(dt)
        s["codes"] = torch.empty(c["rows"], c["cols"] // 2, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty(c["rows"], c["cols"] // 32, dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty_like(s["x"])
        return s
    if c["kind"] in ("ffn", "layer"):
        T, H, I, E, K = c["T"], c["H"], c["I"], c["E"], c["K"]
        s["x"] = _normal(g, T, H).bfloat16()
        s["logits"] = _normal(g, T, E)
        s["w13"], s["w13_s"] = _weights(g, E, 2 * I, H)
        s["w2"], s["w2_s"] = _weights(g, E, H, I)
        if c["kind"] == "ffn":
            _dispatch(s)
        if own:  # the handle that a program keeps: sizes, output buffers and scratch
            s["layer"] = _layer(s)
        return s
    if c["kind"] == "balance":
        T, E, K, B = c["T"], c["E"], c["K"], c["B"]
        s["logits"] = _normal(g, T, E) + _normal(g, E, std=0.7)  # experts of unequal popularity
        if E >= 16:
            s["logits"][:, torch.randint(E, (E // 16,), generator=g, device=DEV)] = -math.inf  # switched off
        s["ids"] = s["logits"].topk(K, dim=1).indices.int()
        cut = torch.sort(torch.randint(0, T + 1, (B - 1,), generator=g, device=DEV)).values.int()
        ends = torch.tensor([0, T], dtype=torch.int32, device=DEV)
        s["seq"] = torch.cat([ends[:1], cut, ends[1:]]).contiguous()
        s["valid"] = (torch.rand(T, generator=g, device=DEV) >= c["pad"]).to(torch.uint8) if c["pad"] else None
        s["dloss"] = 1.0 + 0.1 * _normal(g, B)
        s["loss"] = torch.empty(B, device=DEV)
        s["counts"] = torch.empty(B, E, dtype=torch.int32, device=DEV)
        s["prob_sum"] = torch.empty(B, E, device=DEV)
        s["tokens"] = torch.empty(B, dtype=torch.int32, device=DEV)
        s["dlogits"] = torch.empty(T, E, device=DEV)
        if own:
            import routed_expert_layer_moe_gb300 as moe
            s["p"] = moe.Problem.make(T=T, H=128, I=128, E=E, K=K, layout="contig")
            s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
            s["ws"] = torch.empty(moe.moe_balance_workspace_bytes(s["p"], B), dtype=torch.uint8, device=DEV)
        return s
    T, H, dt = c["T"], c["H"], _dtype(c["dtype"])
    s["x"] = _normal(g, T, H, std=2.0).to(dt)
    s["block"] = _normal(g, T, H, std=0.5).to(dt)
    s["w_post"] = (1.0 + 0.2 * _normal(g, H)).to(dt)
    s["w_pre"] = (1.0 + 0.2 * _normal(g, H)).to(dt)
    s["gate"] = {"none": None, "channel": (0.5 + 0.2 * _normal(g, H)).to(dt),
                 "token": torch.sigmoid(_normal(g, T, 1)).to(dt)}[c["gate"]]
    s["y"], s["xn"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    if c["train"]:
        s["dy"], s["dxn"] = _normal(g, T, H).to(dt), _normal(g, T, H).to(dt)
        s["dx"], s["dblock"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        s["dgate"] = None if s["gate"] is None else torch.empty(s["gate"].shape, device=DEV)
        s["dw_post"], s["dw_pre"] = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
        if own:
            import routed_expert_layer_moe_gb300 as moe
            s["ws"] = torch.empty(moe.moe_block_norm_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
    return s


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _dispatch(s):
    """The grouped MXFP4 activations a dispatch leaves: rows of a slot hold its tokens in ascending order."""
    c = s["case"]
    T, H, E, K = c["T"], c["H"], c["E"], c["K"]
    ids = s.pop("logits").topk(K, dim=1).indices
    order = torch.sort(ids.reshape(-1), stable=True).indices
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    s["masked_m"] = counts.int()
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    most = int(counts.max())
    s["M_max"] = -(-most // 16) * 16  # rows a slot holds at most
    slot = ids.reshape(-1)[order]
    rank = torch.arange(T * K, device=DEV) - s["offsets"].long()[slot]
    row = slot * s["M_max"] + rank if c["layout"] == "masked" else torch.arange(T * K, device=DEV)
    rows = E * s["M_max"] if c["layout"] == "masked" else T * K
    codes, scales = _quantise(s.pop("x").float())
    s["xg"] = torch.zeros(rows, H // 2, dtype=torch.uint8, device=DEV)
    s["xg_s"] = torch.full((rows, H // 32), 127, dtype=torch.uint8, device=DEV)
    s["xg"][row] = codes[order // K]
    s["xg_s"][row] = scales[order // K]


def _layer(s):
    import routed_expert_layer_moe_gb300 as moe
    c = s["case"]
    masked = c.get("layout", "masked") == "masked"
    p = moe.Problem.make(T=c["T"], H=c["H"], I=c["I"], E=c["E"], K=c["K"],
                         M_max=s.get("M_max", c["T"]) if masked else 0, wt="mxfp4",
                         layout="masked" if masked else "contig")
    layer = moe.MoeLayer(p, "bf16", "mxfp4", "bf16", s["w13"], s["w2"], s["w13_s"], s["w2_s"])
    if c["kind"] == "ffn":  # the dispatch has been made: its buffers are the layer's
        layer.xg, layer.xg_s, layer.masked_m, layer.offsets = s["xg"], s["xg_s"], s["masked_m"], s["offsets"]
        layer.yg.zero_()  # padding rows are never written
    return layer


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import routed_expert_layer_moe_gb300 as moe
    c = s["case"]
    if c["kind"] == "mx":
        moe.moe_mx_quantize(s["x"], s["codes"], s["scales"])
        moe.moe_mx_dequantize(s["codes"], s["scales"], s["out"])
        return s["out"]
    if c["kind"] == "ffn":
        s["layer"].ffn()
        return s["layer"].yg
    if c["kind"] == "layer":
        layer = s["layer"]
        out = layer.forward(s["x"], s["logits"], fused=True)
        return {"out": out, "ids": layer.ids}
    if c["kind"] == "balance":
        moe.moe_balance_loss(s["p"], s["logits"], s["ids"], s["valid"], s["seq"], c["score"], 0.01, s["loss"],
                             s["counts"], s["prob_sum"], s["tokens"], s["err"], s["ws"])
        moe.moe_balance_loss_backward(s["p"], s["logits"], s["valid"], s["seq"], c["score"], 0.01, s["counts"],
                                      s["tokens"], s["dloss"], s["dlogits"])
        return {k: s[k] for k in ("loss", "counts", "prob_sum", "tokens", "dlogits")}
    moe.moe_block_norm(s["x"], s["block"], s["gate"], s["w_post"], s["w_pre"], 0.7, EPS, s["y"], s["xn"])
    if not c["train"]:
        return {"y": s["y"], "xn": s["xn"]}
    moe.moe_block_norm_backward(s["x"], s["block"], s["gate"], s["w_post"], s["w_pre"], 0.7, EPS, s["dy"], s["dxn"],
                                s["dx"], s["dblock"], s["dgate"], s["dw_post"], s["dw_pre"], s["ws"])
    return {k: s[k] for k in ("y", "xn", "dx", "dblock", "dgate", "dw_post", "dw_pre")}


# ---- plain forms

def _quantise(x):
    """MXFP4 codes and scales of x (fp32), by elementary operations."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    finite = torch.isfinite(amax)
    e = ((amax.view(torch.int32) >> 23) - 129).clamp(-127, 125)  # floor(log2) - 2; a subnormal's is at most -129
    e = torch.where(finite & (amax > 0), e, torch.zeros_like(e))
    v = b * ((127 - e) << 23).view(torch.float32).unsqueeze(-1)  # times 2^-e, exact
    m = v.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
            + 8 * torch.signbit(b).to(torch.uint8))  # to nearest, ties to the even code
    code = torch.where(finite.unsqueeze(-1), code, torch.zeros_like(code)).flatten(-2)
    scales = torch.where(finite, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def _values(codes, scales, dtype=torch.float32):
    """The values that codes and scales stand for."""
    one = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), device=codes.device, dtype=dtype)
    pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)  # of each byte: the low nibble's, the high's
    v = pair[codes.int()].flatten(-2).unflatten(-1, (-1, 32))
    return (v * _scale(scales, dtype).unsqueeze(-1)).flatten(-2)


def _scale(scales, dtype):
    s = scales.int()
    f = torch.where(s > 0, s << 23, torch.full_like(s, 0x400000)).view(torch.float32).to(dtype)
    return torch.where(s == 255, torch.full_like(f, math.nan), f)


def _plain(s):
    return {"mx": _plain_mx, "ffn": _plain_ffn, "layer": _plain_layer, "balance": _plain_balance,
            "norm": _plain_norm}[s["case"]["kind"]](s)


def _plain_mx(s):
    return _values(*_quantise(s["x"].float())).to(s["x"].dtype)


def _silu_mul(gu):
    g, u = gu.chunk(2, -1)
    return g / (1.0 + torch.exp(-g)) * u


def _plain_ffn(s):
    c, E = s["case"], s["case"]["E"]
    m, off, M = s["masked_m"].long(), s["offsets"].long(), s["M_max"]
    x = _values(s["xg"], s["xg_s"])
    rank = torch.arange(M, device=DEV)
    if c["layout"] == "masked":
        x = x.view(E, M, -1)
    else:
        x = x[(off[:-1, None] + rank).clamp(max=x.shape[0] - 1)]
    gu = torch.bmm(x, _values(s["w13"], s["w13_s"]).transpose(1, 2))
    h = _values(*_quantise(_silu_mul(gu)))
    y = torch.bmm(h, _values(s["w2"], s["w2_s"]).transpose(1, 2))
    if c["layout"] == "masked":
        return torch.where((rank < m[:, None]).unsqueeze(-1), y, torch.zeros_like(y)).flatten(0, 1).bfloat16()
    r = torch.arange(c["T"] * c["K"], device=DEV)
    slot = torch.searchsorted(off[1:].contiguous(), r, right=True)
    return y.flatten(0, 1)[slot * M + r - off[slot]].bfloat16()


def _plain_layer(s):
    K = s["case"]["K"]
    l, ids = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    l, ids = l[:, :K], ids[:, :K]
    w = torch.exp(l - l[:, :1])
    w = w / w.sum(1, keepdim=True)
    x = _values(*_quantise(s["x"].float()))
    gu = torch.matmul(_values(s["w13"][ids], s["w13_s"][ids]), x[:, None, :, None]).squeeze(-1)
    h = _values(*_quantise(_silu_mul(gu)))
    y = torch.matmul(_values(s["w2"][ids], s["w2_s"][ids]), h.unsqueeze(-1)).squeeze(-1)
    return {"out": (y * w.unsqueeze(-1)).sum(1).bfloat16(), "ids": ids.int()}


def _probabilities(l, score):
    """Router scores that sum to one over the experts; a token whose experts are all off has zeros."""
    if score == "softmax":
        top = l.amax(1, keepdim=True)
        a = torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))
    else:
        a = 1.0 / (1.0 + torch.exp(-l))
    z = a.sum(1, keepdim=True)
    return a, a / torch.where(z > 0, z, torch.ones_like(z))


def _balance(l, ids, valid, seq, score, coef, dloss):
    T, E = l.shape
    K, B = ids.shape[1], seq.numel() - 1
    t = torch.arange(T, device=DEV)
    member = (t >= seq[:-1, None]) & (t < seq[1:, None])  # [B, T]
    if valid is not None:
        member = member & (valid != 0)
    inside = member.any(0)
    tokens = member.sum(1)
    a, p = _probabilities(l, score)
    p = torch.where(inside[:, None], p, torch.zeros_like(p))
    prob_sum = torch.matmul(member.to(l.dtype), p)
    b = torch.searchsorted(seq[1:].contiguous(), t.int(), right=True).clamp(max=B - 1)
    counts = torch.zeros(B * E, dtype=torch.int32, device=DEV)
    counts.index_add_(0, (b[:, None] * E + ids).reshape(-1), inside[:, None].int().expand(T, K).reshape(-1))
    counts = counts.view(B, E)
    n = tokens.clamp(min=1).to(l.dtype)
    scale = coef * E / (K * n * n)
    loss = scale * (counts * prob_sum).sum(1)
    # the gradient of a score: scale * counts, less its mean under p (scores that sum to one)
    v = (counts - (counts.sum(1, keepdim=True).to(l.dtype) / E)) * (scale * dloss)[:, None]
    v = v[b]
    d = p * (v - (v * p).sum(1, keepdim=True))
    if score == "sigmoid":
        d = d * (1.0 - a)
    return {"loss": loss, "counts": counts, "prob_sum": prob_sum, "tokens": tokens.int(), "dlogits": d}


def _plain_balance(s):
    return _balance(s["logits"], s["ids"], s["valid"], s["seq"], s["case"]["score"], 0.01, s["dloss"])


def _plain_norm(s):
    x, b, wp, wn = (s[k].float() for k in ("x", "block", "w_post", "w_pre"))
    H, rs, kind, dt = x.shape[1], 0.7, s["case"]["gate"], s["x"].dtype
    g = 1.0 if s["gate"] is None else s["gate"].float()
    rb = torch.rsqrt((b * b).mean(1, keepdim=True) + EPS)
    bn = b * rb
    y = x + rs * g * (bn * wp)
    ry = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
    yn = y * ry
    out = {"y": y.to(dt), "xn": (yn * wn).to(dt)}
    if not s["case"]["train"]:
        return out
    dy, dxn = s["dy"].float(), s["dxn"].float()
    q = dxn * wn
    dx = dy + ry * (q - yn * (q * yn).mean(1, keepdim=True))
    q = rs * g * dx * wp
    db = rb * (q - bn * (q * bn).mean(1, keepdim=True))
    dgate = None if kind == "none" else (rs * dx * bn * wp).sum(0 if kind == "channel" else 1, keepdim=kind == "token")
    return {**out, "dx": dx.to(dt), "dblock": db.to(dt), "dgate": dgate, "dw_post": (rs * g * dx * bn).sum(0),
            "dw_pre": (dxn * yn).sum(0)}


# ---------------------------------------------------------------------------------------------- 64 bits

def _exact_mx(x):
    """The values that the MXFP4 form of x stands for, from the definition, in 64 bits."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    top = b.abs().max(-1, keepdim=True).values
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e))
    e = torch.where(top > 0, (e - 2).clamp(-127, 125), torch.zeros_like(e))
    unit = torch.exp2(e)
    m = (b / unit).abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
    v = (torch.round(m / step) * step).clamp(max=6.0)  # torch.round takes ties to the even integer
    return (torch.sign(b) * v * unit).reshape(x.shape)


def _exact_expert(x, s, e):
    gu = x @ _values(s["w13"][e], s["w13_s"][e], torch.float64).T
    I = gu.shape[1] // 2
    h = _exact_mx(gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:])
    return h @ _values(s["w2"][e], s["w2_s"][e], torch.float64).T


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "mx":
        return _exact_mx(s["x"])
    if c["kind"] == "ffn":
        x = _values(s["xg"], s["xg_s"], torch.float64)
        y = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
        for e, (m, o) in enumerate(zip(s["masked_m"].tolist(), s["offsets"].tolist())):
            at = e * s["M_max"] if c["layout"] == "masked" else o
            if m:
                y[at:at + m] = _exact_expert(x[at:at + m], s, e)
        return y
    if c["kind"] == "layer":
        l = s["logits"].double()
        out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV)
        x = _exact_mx(s["x"])
        for t in range(c["T"]):
            ids = sorted(range(c["E"]), key=lambda e: (-float(l[t, e]), e))[:c["K"]]
            w = torch.softmax(l[t, ids], 0)
            for k, e in enumerate(ids):
                out[t] += w[k] * _exact_expert(x[t:t + 1], s, e)[0]
        return {"out": out, "ids": None}
    if c["kind"] == "balance":
        return _exact_balance(s)
    return _exact_norm(s)


def _exact_balance(s):
    """Segment by segment, the gradient by automatic differentiation of the loss in 64 bits."""
    c = s["case"]
    E, K = c["E"], c["K"]
    loss, sums = [], []
    grad = torch.zeros(s["logits"].shape, dtype=torch.float64, device=DEV)
    seq = s["seq"].tolist()
    for b in range(c["B"]):
        rows = torch.arange(seq[b], seq[b + 1], device=DEV)
        if s["valid"] is not None:
            rows = rows[s["valid"][rows] != 0]
        n = len(rows)
        if n == 0:
            loss.append(torch.zeros((), dtype=torch.float64, device=DEV))
            sums.append(torch.zeros(E, dtype=torch.float64, device=DEV))
            continue
        l = s["logits"][rows].double().requires_grad_()
        f = torch.bincount(s["ids"][rows].reshape(-1).long(), minlength=E).double() * (E / (K * n))
        p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
        p = p / p.sum(1, keepdim=True)
        one = 0.01 * (f * p.mean(0)).sum()
        (one * s["dloss"][b].double()).backward()
        grad[rows] = l.grad
        loss.append(one.detach())
        sums.append(p.detach().sum(0))
    return {"loss": torch.stack(loss), "counts": None, "prob_sum": torch.stack(sums), "tokens": None, "dlogits": grad}


def _exact_norm(s):
    c, rs = s["case"], 0.7
    leaf = {k: s[k].double().requires_grad_() for k in ("x", "block", "w_post", "w_pre")}
    gate = None if s["gate"] is None else s["gate"].double().requires_grad_()

    def rms(v):
        return v / torch.sqrt(v.square().sum(1, keepdim=True) / v.shape[1] + EPS)

    branch = rms(leaf["block"]) * leaf["w_post"]
    y = leaf["x"] + rs * (branch if gate is None else gate * branch)
    xn = rms(y) * leaf["w_pre"]
    out = {"y": y.detach(), "xn": xn.detach()}
    if not c["train"]:
        return out
    torch.autograd.backward([y, xn], [s["dy"].double(), s["dxn"].double()])
    return {**out, "dx": leaf["x"].grad, "dblock": leaf["block"].grad, "dgate": None if gate is None else gate.grad,
            "dw_post": leaf["w_post"].grad, "dw_pre": leaf["w_pre"].grad}
