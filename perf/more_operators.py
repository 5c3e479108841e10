"""Cases that measure what trains the experts of the MoE layer, each with its plain form.

  ckpt  an activation checkpoint in 8 bits and back (moe_fp8_quantize, moe_fp8_dequantize)
  up    the gate/up product of a training pass, which keeps its results for the gradient in 8 bits
        (moe_grouped_swiglu_gemm_save)
  back  the gradient of the layer from its output to its input, its router's logits and its weights, on that
        checkpoint (moe_combine_backward, moe_grouped_ffn_backward, moe_permute_backward, moe_route_backward)

A checkpoint holds, per group of 128 values of a row (the last group of a row may be shorter), E4M3 codes and one fp32
scale: s = largest magnitude / 448 (1 where that is zero), code = E4M3(x / s), the nearest to the quotient before any
other rounding, ties to even.

The layer: rows of an expert e are x of its tokens; (g, u) = x W13[e]^T, h = silu(g) u, y = h W2[e]^T, and a token's
output is the sum of its K experts' y with the router's weights w (softmax over the K chosen logits), plus that of
the shared expert where there is one.  The gradient takes g and u as the checkpoint holds them.

`run` computes the plain form with elementary torch operations in 32 bits where `own` is false, and calls the
library where it is true."""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
GROUP = 128


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode-sized batch's layer output, kept for a gradient
        {"name": "ckpt_small", "kind": "ckpt", "rows": 128, "cols": 7168, "dtype": "bf16"},
        # a training step's layer output: 8192 tokens
        {"name": "ckpt_step", "kind": "ckpt", "rows": 8192, "cols": 4096, "dtype": "bf16"},
        # fp32 rows whose last group is short and that start at any multiple of 4 bytes
        {"name": "ckpt_odd_rows", "kind": "ckpt", "rows": 4001, "cols": 6290, "dtype": "f32"},
        # few tokens, small experts: the latency of one launch
        {"name": "up_small", "kind": "up", "T": 48, "H": 512, "I": 384, "E": 8, "K": 2, "shared": 0,
         "layout": "masked", "skew": 0.7},
        # Mixtral-8x7B-shaped experts, 4096 tokens: bound by the tensor cores
        {"name": "up_8_experts", "kind": "up", "T": 4096, "H": 4096, "I": 14336, "E": 8, "K": 2, "shared": 0,
         "layout": "contig", "skew": 0.0},
        # the prefill workload's experts: 8.6 GB of weights over 160 rows each
        {"name": "up_512_experts", "kind": "up", "T": 8192, "H": 4096, "I": 1024, "E": 512, "K": 10, "shared": 0,
         "layout": "contig", "skew": 0.0},
        # a small batch through small experts: each launch's latency counts
        {"name": "back_small", "kind": "back", "T": 32, "H": 512, "I": 256, "E": 8, "K": 2, "shared": 0,
         "layout": "masked", "skew": 0.7},
        # sizes that divide no tile, a shared expert, experts of very different popularity
        {"name": "back_odd_shared", "kind": "back", "T": 777, "H": 1152, "I": 640, "E": 24, "K": 3, "shared": 1,
         "layout": "masked", "skew": 1.5},
        # many small experts with ragged groups: 65536 rows over 64 experts
        {"name": "back_64_experts", "kind": "back", "T": 8192, "H": 2048, "I": 1024, "E": 64, "K": 8, "shared": 0,
         "layout": "contig", "skew": 0.7},
        # Mixtral-8x7B-shaped experts, a micro-batch of 4096 tokens
        {"name": "back_8_experts", "kind": "back", "T": 4096, "H": 4096, "I": 14336, "E": 8, "K": 2, "shared": 0,
         "layout": "contig", "skew": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    """A multiple of m, spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, _log(rng, lo, hi) // m * m))


def draw(rng):
    kind = rng.choice(["ckpt", "up", "up", "back", "back", "back"])
    if kind == "ckpt":
        while True:
            c = {"kind": kind, "rows": _log(rng, 1, 65536), "cols": _log(rng, 1, 16384),
                 "dtype": rng.choice(["bf16", "f32"])}
            if rng.random() < 0.6:
                c["cols"] = max(128, c["cols"] // 128 * 128)
            if c["rows"] * c["cols"] <= 4001 * 6290:
                return c
    while True:
        E = _log(rng, 1, 512 if kind == "up" else 128)
        c = {"kind": kind, "T": _log(rng, 1, 8192), "H": _mult(rng, 128, 7168, 128), "I": _mult(rng, 128, 14336, 128),
             "E": E, "K": rng.randint(1, min(E, 10)), "shared": int(rng.random() < 0.25),
             "layout": rng.choice(["masked", "contig"]), "skew": rng.choice([0.0, 0.7, 1.5])}
        rows, w = c["T"] * (c["K"] + c["shared"]), c["H"] * c["I"]
        most = 8192 * 4096 * 14336 // (1 if kind == "back" else 2)
        weights = (E + c["shared"]) * w <= (512 * 4096 * 1024 if kind == "up" else 8 * 4096 * 14336)
        # the plain form holds every expert's rows at the most popular one's number
        most_rows = min(c["T"], {0.0: 2, 0.7: 8, 1.5: E}[c["skew"]] * c["T"] * c["K"] // E + 64)
        if c["shared"] or c["layout"] == "masked":
            most_rows = c["T"]
        padded = (E + c["shared"]) * most_rows * (c["H"] + 2 * c["I"]) <= 1 << 31
        if rows * w <= most and weights and padded:
            return c


def work(case):
    c = case
    if c["kind"] == "ckpt":
        n, es = c["rows"] * c["cols"], 2 if c["dtype"] == "bf16" else 4
        # the values, the codes and scales that are kept, the values they stand for
        return {"bytes": n * (es + 1) + 4 * c["rows"] * -(-c["cols"] // GROUP) + n * es, "flops": 0}
    T, H, I, E, K, S = (c[k] for k in ("T", "H", "I", "E", "K", "shared"))
    rows = T * (K + S)
    touched = E * (1.0 - (1.0 - K / E) ** T) + S
    if c["kind"] == "up":
        return {"bytes": touched * 2 * I * H * 2 + rows * H * 2 + rows * I * 2 + rows * 2 * I * (1 + 4 / GROUP),
                "flops": 4.0 * rows * H * I}
    weights = touched * 3 * H * I * 2 + (E + S) * 3 * H * I * 2  # read, and their gradients written
    acts = rows * H * 4 + rows * 2 * I * (1 + 4 / GROUP) + T * H * 4 + T * E * 4
    return {"bytes": weights + acts, "flops": 12.0 * rows * H * I}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * std


def _weights(g, n, rows, cols):
    w = torch.empty(n, rows, cols, dtype=torch.bfloat16, device=DEV)
    for e in range(n):
        w[e] = _normal(g, rows, cols, std=0.02)
    return w


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["kind"] == "ckpt":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["x"] = (_normal(g, c["rows"], c["cols"]) * torch.exp(_normal(g, c["rows"], 1))).to(dt)
        s["codes"] = torch.empty(c["rows"], c["cols"], dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty(c["rows"], -(-c["cols"] // GROUP), device=DEV)
        s["out"] = torch.empty_like(s["x"])
        return s
    T, H, I, E, K, S = (c[k] for k in ("T", "H", "I", "E", "K", "shared"))
    logits = _normal(g, T, E) + _normal(g, E, std=1.0) * c["skew"]
    _dispatch(s, logits)
    rows = s["rows"]
    x = _normal(g, T, H).bfloat16()
    s["xg"] = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
    s["xg"][s["row_of"].long()] = x[:, None]
    s["w13"] = _weights(g, E + S, 2 * I, H)
    s["gu"] = torch.zeros(rows, 2 * I, dtype=torch.uint8, device=DEV)
    s["gu_s"] = torch.ones(rows, 2 * I // GROUP, device=DEV)
    if c["kind"] == "back":
        s["w2"] = _weights(g, E + S, H, I)
        used = s["row_of"].reshape(-1).long()
        for a in range(0, used.numel(), 4096):  # what x of unit variance gives through weights of 0.02
            part = used[a:a + 4096]
            s["gu"][part], s["gu_s"][part] = _quantise(_normal(g, part.numel(), 2 * I, std=0.02 * math.sqrt(H)))
        s["yg"] = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
        s["yg"][used] = _normal(g, used.numel(), H, std=0.5).bfloat16()
        s["dout"] = _normal(g, T, H, std=0.1).bfloat16()
    else:
        s["values"] = torch.zeros(rows, 2 * I, dtype=torch.bfloat16, device=DEV)
    if own:  # the handle that a program keeps: sizes, output buffers and scratch
        s["layer"] = _layer(s)
    return s


def _dispatch(s, logits):
    """The routing and the layout that the layer's first steps leave: rows of a slot hold its tokens in ascending
    order; the shared expert's slot is the last one and holds every token."""
    c = s["case"]
    T, E, K, S = (c[k] for k in ("T", "E", "K", "shared"))
    top = logits.topk(K, dim=1)
    s["ids"], s["w"] = top.indices.int(), torch.softmax(top.values, 1)
    slots = top.indices
    if S:
        slots = torch.cat([slots, torch.full((T, 1), E, device=DEV)], 1)
    flat = slots.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E + S)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    s["most"] = max(1, int(counts.max()))
    s["M_max"] = T  # rows a slot of the masked layout holds at most
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(flat.numel(), device=DEV) - offsets[flat[order]]
    base = flat * s["M_max"] if c["layout"] == "masked" else offsets[flat]
    s["rows"] = (E + S) * s["M_max"] if c["layout"] == "masked" else flat.numel()
    s["masked_m"], s["offsets"] = counts.int(), offsets.int()
    s["row_of"] = (base + rank).view(T, K + S).int()
    s["src_of"] = torch.full((s["rows"],), -1, dtype=torch.int32, device=DEV)
    s["src_of"][s["row_of"].long()] = torch.arange(T, device=DEV, dtype=torch.int32)[:, None]


def _layer(s):
    import routed_expert_layer_moe_gb300 as moe
    c = s["case"]
    masked = c["layout"] == "masked"
    p = moe.Problem.make(T=c["T"], H=c["H"], I=c["I"], E=c["E"], K=c["K"], M_max=s["M_max"] if masked else 0,
                         has_shared=c["shared"], wt="bf16", layout=c["layout"])
    layer = moe.MoeLayer(p, "bf16", "bf16", "bf16", s["w13"], s.get("w2"), train=True)
    # the routing and the dispatch have been made: their buffers are the layer's
    for k in ("ids", "w", "masked_m", "offsets", "row_of", "src_of", "xg", "gu", "gu_s"):
        setattr(layer, k, s[k])
    if "yg" in s:
        layer.yg = s["yg"]
    layer.hg.zero_()  # padding rows are never written
    return layer


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import routed_expert_layer_moe_gb300 as moe
    c = s["case"]
    if c["kind"] == "ckpt":
        moe.moe_fp8_quantize(s["x"], s["codes"], s["scales"])
        moe.moe_fp8_dequantize(s["codes"], s["scales"], s["out"])
        return s["out"]
    layer = s["layer"]
    if c["kind"] == "up":
        layer.swiglu_save()
        moe.moe_fp8_dequantize(layer.gu, layer.gu_s, s["values"])
        return {"h": layer.hg, "gu": s["values"]}
    dx, dlogits, dw13, dw2 = layer.backward(s["dout"])
    return {"dx": dx, "dlogits": dlogits, "dw13": dw13, "dw2": dw2}


# ---- plain forms

def _e4m3(m):
    """The nearest E4M3 magnitude of m >= 0 (64 bits: a quotient next to a border must not reach it by being rounded),
    ties to the even code, and the number of steps from zero's binade or its own that it is."""
    e = ((m.view(torch.int64) >> 52) - 1023).clamp(-6, 8)
    step = ((e - 3 + 1023) << 52).view(torch.float64)  # distance of neighbours: 2^(e - 3)
    units = torch.round(m / step)
    return (units * step).clamp(max=E4M3_MAX), units.int(), e.int()


def _groups(x):
    """x [rows, cols] as [rows, groups, 128], the last group filled up with zeros."""
    rows, cols = x.shape
    n = -(-cols // GROUP)
    if cols % GROUP:
        x = torch.cat([x, x.new_zeros(rows, n * GROUP - cols)], 1)
    return x.view(rows, n, GROUP)


def _scales(b):
    amax = b.abs().amax(-1)
    return torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))


def _round8(x):
    """What the checkpoint of x [rows, cols] (fp32) stands for."""
    b = _groups(x)
    sc = _scales(b).unsqueeze(-1)
    v = b.double() / sc
    return (torch.where(v < 0, -1.0, 1.0) * _e4m3(v.abs())[0].float() * sc).flatten(1)[:, :x.shape[1]]


def _quantise(x):
    """Codes (a byte each) and scales of x [rows, cols], cols a multiple of 128."""
    b = _groups(x)
    sc = _scales(b)
    v = b.double() / sc.unsqueeze(-1)
    _, units, e = _e4m3(v.abs())
    # units: 8..16, or 0..8 below the smallest normal; 16 of one binade are 8 of the next, and their codes follow on
    code = (units + 8 * (e + 6)).clamp(max=126) + 128 * torch.signbit(v).int()
    return code.to(torch.uint8).flatten(1), sc


def _values(codes, scales, dtype=torch.float32):
    """The values that codes [..., cols] and scales [..., cols / 128] stand for."""
    i = torch.arange(256, device=codes.device)
    e, m = (i >> 3) & 15, (i & 7).to(dtype)
    one = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).to(dtype)), m * 2.0 ** -9)
    one = torch.where(i >= 128, -one, one)
    v = one[codes.int()].unflatten(-1, (-1, GROUP)) * scales.to(dtype).unsqueeze(-1)
    return v.flatten(-2)


def _plain(s):
    return {"ckpt": _plain_ckpt, "up": _plain_up, "back": _plain_back}[s["case"]["kind"]](s)


def _plain_ckpt(s):
    return _round8(s["x"].float()).to(s["x"].dtype)


def _slots(s):
    """Rows of the grouped buffer by slot and rank [slots, most], and which of them hold a token."""
    c, m = s["case"], s["masked_m"].long()
    n = m.numel()
    rank = torch.arange(s["most"], device=DEV)
    base = torch.arange(n, device=DEV) * s["M_max"] if c["layout"] == "masked" else s["offsets"].long()[:-1]
    return (base[:, None] + rank).clamp(max=s["rows"] - 1), rank < m[:, None]


def _places(s):
    """Where in [slots * most] each record of each token is."""
    c, row = s["case"], s["row_of"].long()
    slot = s["ids"].long()
    if c["shared"]:
        slot = torch.cat([slot, torch.full_like(slot[:, :1], c["E"])], 1)
    base = slot * s["M_max"] if c["layout"] == "masked" else s["offsets"].long()[slot]
    return slot * s["most"] + row - base


def _back_to_rows(s, v):
    """v [slots, most, cols] in the grouped buffer's rows, zeros in its padding."""
    out = v.new_zeros(s["rows"], v.shape[-1])
    out[s["row_of"].long()] = v.flatten(0, 1)[_places(s)]
    return out


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _plain_up(s):
    at, live = _slots(s)
    x = torch.where(live.unsqueeze(-1), s["xg"][at].float(), 0.0)
    gu = torch.bmm(x, s["w13"].float().transpose(1, 2))
    g, u = gu.chunk(2, -1)
    return {"h": _back_to_rows(s, g * _sigmoid(g) * u).bfloat16(), "gu": _round8(_back_to_rows(s, gu)).bfloat16()}


def _plain_back(s):
    c = s["case"]
    T, E, K = c["T"], c["E"], c["K"]
    at, live = _slots(s)
    live = live.unsqueeze(-1)
    dout, w, row = s["dout"].float(), s["w"], s["row_of"].long()
    # the combine: dy = w dout by record, dw = dout . y
    dw = (dout[:, None] * s["yg"][row[:, :K]].float()).sum(-1)
    dlogits = torch.zeros(T, E, device=DEV)
    dlogits.scatter_(1, s["ids"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    wr = torch.ones(s["rows"], device=DEV)
    wr[row[:, :K]] = w
    dy = torch.where(live, dout[s["src_of"].clamp(min=0).long()[at]] * wr[at].unsqueeze(-1), 0.0)
    # the experts
    g, u = torch.where(live, _values(s["gu"][at], s["gu_s"][at]), 0.0).chunk(2, -1)
    sg = _sigmoid(g)
    dh = torch.bmm(dy, s["w2"].float())
    dw2 = torch.bmm(dy.transpose(1, 2), g * sg * u).bfloat16()
    dgu = torch.cat([dh * u * (sg * (1.0 + g * (1.0 - sg))), dh * (g * sg)], -1)
    x = torch.where(live, s["xg"][at].float(), 0.0)
    dw13 = torch.bmm(dgu.transpose(1, 2), x).bfloat16()
    dx = torch.bmm(dgu, s["w13"].float()).flatten(0, 1)[_places(s)].sum(1)
    return {"dx": dx.bfloat16(), "dlogits": dlogits, "dw13": dw13, "dw2": dw2}


# ---------------------------------------------------------------------------------------------- 64 bits

def _exact_round8(x):
    """The values that the checkpoint of x (fp64) stands for, from the definition: scales are fp32."""
    out = torch.empty_like(x)
    for a in range(0, x.shape[1], GROUP):
        b = x[:, a:a + GROUP]
        sc = (b.abs().max(1, keepdim=True).values.float() / E4M3_MAX).double()
        sc = torch.where(sc > 0, sc, torch.ones_like(sc))
        v = b / sc
        m = v.abs()
        e = torch.floor(torch.log2(m.clamp(min=2.0 ** -6)))
        step = torch.exp2(e.clamp(max=8) - 3)
        out[:, a:a + GROUP] = torch.sign(v) * (torch.round(m / step) * step).clamp(max=E4M3_MAX) * sc
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "ckpt":
        return _exact_round8(s["x"].double())
    T, H, I, E, K, S = (c[k] for k in ("T", "H", "I", "E", "K", "shared"))
    counts, starts = s["masked_m"].tolist(), s["offsets"].tolist()
    if c["layout"] == "masked":
        starts = [e * s["M_max"] for e in range(E + S)]
    part = [(e, slice(starts[e], starts[e] + counts[e])) for e in range(E + S) if counts[e]]
    if c["kind"] == "up":
        h = torch.zeros(s["rows"], I, dtype=torch.float64, device=DEV)
        kept = torch.zeros(s["rows"], 2 * I, dtype=torch.float64, device=DEV)
        for e, r in part:
            gu = s["xg"][r].double() @ s["w13"][e].double().T
            h[r] = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
            kept[r] = _exact_round8(gu)
        return {"h": h, "gu": kept}
    dout, w = s["dout"].double(), s["w"].double()
    dw13 = torch.zeros(E + S, 2 * I, H, dtype=torch.float64, device=DEV)
    dw2 = torch.zeros(E + S, H, I, dtype=torch.float64, device=DEV)
    dxg = torch.zeros(s["rows"], H, dtype=torch.float64, device=DEV)
    weight = torch.ones(s["rows"], 1, dtype=torch.float64, device=DEV)
    for k in range(K):
        weight[s["row_of"][:, k].long(), 0] = w[:, k]
    for e, r in part:
        gu = _values(s["gu"][r], s["gu_s"][r], torch.float64).requires_grad_()
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        dy = weight[r] * dout[s["src_of"][r].long()]
        dgu, = torch.autograd.grad(h, gu, dy @ s["w2"][e].double())
        dw2[e] = dy.T @ h.detach()
        dw13[e] = dgu.T @ s["xg"][r].double()
        dxg[r] = dgu @ s["w13"][e].double()
    dx = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for k in range(K + S):
        dx += dxg[s["row_of"][:, k].long()]
    dlogits = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    dw = torch.stack([(dout * s["yg"][s["row_of"][:, k].long()].double()).sum(1) for k in range(K)], 1)
    jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
    dlogits.scatter_add_(1, s["ids"].long(), torch.einsum("tij,tj->ti", jac, dw))
    return {"dx": dx, "dlogits": dlogits, "dw13": dw13, "dw2": dw2}
