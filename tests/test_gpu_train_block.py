"""Training passes as a program makes them: the whole block, streams, graphs, replicas, dropped records, large sizes."""
import importlib.util
import os

import pytest
import torch

import operator_reference as ref
import routed_expert_layer_moe_gb300 as moe
import train_reference as tref
from test_gpu_train import HALF, d, layer_reference, make_layer, sums

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def example():
    from routed_expert_layer_moe_gb300 import build
    build.build()
    torch.cuda.init()
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def off(got, want):
    return float((d(got) - want).norm() / want.norm())


def block_objective(block, w, x, ids, dy, dxn, dloss):
    """What the example's gradients are of, in 64 bits, with the routing's choice held: a function of x and the weights."""
    p = block.p
    xn = ref.block_norm(x, None, None, None, w["w_pre"], 1.0, 1e-6)[1]
    logits = xn @ w["w_g"]
    weight = tref.route_weights(logits, ids, "softmax", True, 1.0)
    out = torch.zeros_like(x)
    for e in range(p.E):
        t, k = (ids == e).nonzero(as_tuple=True)
        if len(t):
            gu = xn[t] @ w["w13"][e].T
            y = tref.swiglu(gu[:, :p.I], gu[:, p.I:]) @ w["w2"][e].T
            out = out.index_add(0, t, weight[t, k][:, None] * y)
    y, xn_next = ref.block_norm(x, out, w["gate"], w["w_post"], w["w_next"], 1.0, 1e-6)
    n = torch.bincount(ids.flatten().long(), minlength=p.E).double()
    prob = torch.softmax(logits, 1).sum(0)
    balance = 0.01 * p.E / (p.K * p.T ** 2) * (n * prob).sum()
    return (dy * y).sum() + (dxn * xn_next).sum() + dloss * balance


def test_block(example):
    T, H, I, E, K = 70, 256, 384, 5, 2
    block, w_g = example.make_block(T, H, I, E, K)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    dy, dxn = (torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(2))
    dloss = torch.tensor([100.0], device="cuda")
    y, xn_next, logits = example.forward(block, w_g, x)
    plain = moe.MoeLayer(block.p, "bf16", "bf16", "bf16", block.layer.w13, block.layer.w2)
    o = plain.forward(block.xn, logits)
    assert off(block.layer.out, d(o)) <= 2 * HALF
    dx, grads = example.backward(block, w_g, x, logits, dy, dxn, dloss)
    torch.cuda.synchronize()
    assert int(block.layer.err) == 0
    w = {"w_pre": block.w_pre, "w_g": w_g, "w13": block.layer.w13, "w2": block.layer.w2, "gate": block.gate,
         "w_post": block.w_post, "w_next": block.w_next}
    w = {k: d(v).requires_grad_() for k, v in w.items()}
    xl = d(x).requires_grad_()
    args = (block.layer.ids.cpu(), d(dy), d(dxn), float(dloss))
    block_objective(block, w, xl, *args).backward()
    # The checkpoint holds g and u to 2^-4 of themselves each: h and the slopes are off by 2^-3 of their size at most, in
    # norm, and everything behind them; what is not behind them has bf16 roundings alone.
    for name, got in {"x": dx, **grads}.items():
        want = (xl if name == "x" else w[name]).grad
        assert off(got, want) <= (8 * HALF if name in ("gate", "w_post", "w_next") else 2.0 ** -3), name
    # the reference itself, against differences along a random direction of everything
    with torch.no_grad():
        v = {k: torch.randn(t.shape, generator=g).double() * t.abs().mean() for k, t in w.items()}
        vx = torch.randn(x.shape, generator=g).double()
        s = 1e-5
        f = lambda sign: block_objective(block, {k: t + sign * s * v[k] for k, t in w.items()}, xl + sign * s * vx, *args)  # noqa: E731
        slope = (f(1) - f(-1)) / (2 * s)
    along = sum((w[k].grad * v[k]).sum() for k in w) + (xl.grad * vx).sum()
    assert abs(slope - along) <= 1e-6 * abs(along) + 1e-6


def test_example_runs(example, capsys):
    example.main()
    assert capsys.readouterr().out.count("loss") == 3


def test_kept_output(example):
    """leave_backward() on the 8-bit checkpoint of an output that another pass has overwritten."""
    block, w_g = example.make_block(33, 256, 128, 4, 2)
    x, x2, dy, dxn = (torch.randn(33, 256, device="cuda").bfloat16() for _ in range(4))
    example.forward(block, w_g, x)
    out, kept = block.layer.out.clone(), block.keep_out()
    example.forward(block, w_g, x2)
    codes, scales = tref.fp8_quantize(out.cpu().double().numpy())
    value = torch.from_numpy(tref.fp8_values(codes, scales)).float().bfloat16().cuda()
    for a, b in zip(block.leave_backward(x, dy, dxn, out=kept), block.leave_backward(x, dy, dxn, out=value)):
        assert torch.equal(a, b)


def test_captured_and_replayed(example):
    block, w_g = example.make_block(50, 256, 256, 6, 2)
    xs = [torch.randn(50, 256, device="cuda").bfloat16() for _ in range(3)]
    x, dy, dxn, dloss = xs[0].clone(), xs[1], xs[2], torch.ones(1, device="cuda")

    def step():
        y, xn_next, logits = example.forward(block, w_g, x)
        dx, grads = example.backward(block, w_g, x, logits, dy, dxn, dloss)
        return [y, dx, *grads.values()]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for other in (xs[2], xs[1]):
        x.copy_(other)
        for t in got:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got_now = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(got_now, step()))


def test_two_layers_on_two_streams():
    """Training passes of two layers on the same weights, at once on two streams, give what they give in turn."""
    a, r = make_layer(300, 512, 384, 6, 2)
    b = moe.MoeLayer(a.p, "bf16", "bf16", "bf16", a.w13, a.w2, train=True)
    data = [(r(300, 512).bfloat16(), r(300, 6), r(300, 512).bfloat16()) for _ in range(2)]

    def one(layer, x, logits, dout, stream=None):
        layer.forward(x, logits, stream, save=True)
        return layer.backward(dout, stream=stream)

    want = [[t.clone() for t in one(layer, *v)] for layer, v in zip((a, b), data)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        torch.cuda.synchronize()
        got = [one(layer, *v, stream=s) for layer, v, s in zip((a, b), data, streams)]
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(x, y))
    assert int(a.err) == int(b.err) == 0


def test_accumulating_micro_batches():
    a, r = make_layer(64, 256, 256, 4, 2)
    b = moe.MoeLayer(a.p, "bf16", "bf16", "bf16", a.w13, a.w2, train=True)
    dw13, dw2 = (torch.zeros(t.shape, device="cuda") for t in (a.w13, a.w2))
    data = [(r(64, 256).bfloat16(), r(64, 4), r(64, 256).bfloat16()) for _ in range(2)]
    for layer, (x, logits, _) in zip((a, b), data):
        layer.forward(x, logits, save=True)
    single = [layer.backward(v[2], torch.empty_like(dw13), torch.empty_like(dw2)) for layer, v in zip((a, b), data)]
    for layer, v in zip((a, b), data):
        layer.backward(v[2], dw13, dw2, accumulate=True)
    assert torch.equal(dw13, single[0][2] + single[1][2]) and torch.equal(dw2, single[0][3] + single[1][3])
    dx, dlogits, none13, none2 = a.backward(data[0][2], weights=False)
    assert none13 is None and none2 is None and torch.equal(dx, single[0][0]) and torch.equal(dlogits, single[0][1])
    for bad in (dict(accumulate=True), dict(dw13=dw13, accumulate=True), dict(weights=False, accumulate=True)):
        with pytest.raises(ValueError):
            a.backward(data[0][2], **bad)
    with pytest.raises(moe.MoeError):  # bf16 gradients are not added to
        a.backward(data[0][2], torch.zeros_like(a.w13), torch.zeros_like(a.w2), accumulate=True)
    plain = moe.MoeLayer(a.p, "bf16", "bf16", "bf16", a.w13, a.w2)
    for call in (lambda: plain.backward(data[0][2]), lambda: plain.swiglu_save(),
                 lambda: plain.forward(*data[0][:2], save=True)):
        with pytest.raises(ValueError, match="train"):
            call()


def test_replicas_have_their_own_gradients():
    E, P = 4, 7
    p2l = torch.tensor([0, 1, 2, 3, 1, 1, 3], dtype=torch.int32, device="cuda")
    one, r = make_layer(90, 256, 128, E, 2)
    x, logits, dout = r(90, 256).bfloat16(), r(90, E), r(90, 256).bfloat16()
    one.forward(x, logits, save=True)
    want = one.backward(dout, torch.empty(one.w13.shape, device="cuda"), torch.empty(one.w2.shape, device="cuda"))
    p = moe.Problem.make(T=90, H=256, I=128, E=E, K=2, P=P, layout="contig")
    many = moe.MoeLayer(p, "bf16", "bf16", "bf16", one.w13[p2l.long()].contiguous(), one.w2[p2l.long()].contiguous(),
                        phys_to_log=p2l, train=True)
    many.forward(x, logits, save=True)
    got = many.backward(dout, torch.empty(many.w13.shape, device="cuda"), torch.empty(many.w2.shape, device="cuda"))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for g, w, terms in zip(got[2:], want[2:], (90, 90)):
        per_expert = torch.zeros_like(w).index_add_(0, p2l.long(), g)
        # the same terms in groups of another order; sums of positive and negative terms: bounded by their norm's
        assert off(per_expert, d(w)) <= 64 * sums(terms)


def test_dropped_records():
    """Slots that overflow: records without a place have no part in any gradient."""
    layer, r = make_layer(60, 256, 128, 3, 2)
    p = moe.Problem.make(T=60, H=256, I=128, E=3, K=2, M_max=24, layout="masked")
    layer = moe.MoeLayer(p, "bf16", "bf16", "bf16", layer.w13, layer.w2, train=True)
    x, logits, dout = r(60, 256).bfloat16(), r(60, 3), r(60, 256).bfloat16()
    layer.forward(x, logits, save=True)
    grads = layer.backward(dout)
    torch.cuda.synchronize()
    assert int(layer.err) == moe.MOE_FLAG_OVERFLOW and bool((layer.row_of < 0).any())
    layer.masked_m.clamp_(max=24)  # for the reference's list of rows
    for got, v in zip(grads, layer_reference(layer, dout, logits=logits)):
        assert off(got, v) <= 4 * HALF


def test_empty_batch():
    for layout in ("masked", "contig"):
        g = torch.Generator(device="cuda").manual_seed(0)
        p = moe.Problem.make(T=0, H=128, I=128, E=3, K=2, M_max=8 if layout == "masked" else 0, layout=layout)
        w13, w2 = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((3, 256, 128), (3, 128, 128)))
        layer = moe.MoeLayer(p, "bf16", "bf16", "bf16", w13, w2, train=True)
        x, logits = torch.empty(0, 128, device="cuda").bfloat16(), torch.empty(0, 3, device="cuda")
        assert layer.forward(x, logits, save=True).shape == (0, 128)
        dx, dlogits, dw13, dw2 = layer.backward(x)
        torch.cuda.synchronize()
        assert dx.shape == (0, 128) and dlogits.shape == (0, 3) and not dw13.any() and not dw2.any()
        assert int(layer.err) == 0


def test_outputs_at_16_bytes():
    """Buffers that start 16 bytes into a 32-byte sector take the narrower stores and give the same bits."""
    layer, r = make_layer(150, 256, 384, 5, 2)
    x, logits, dout = r(150, 256).bfloat16(), r(150, 5), r(150, 256).bfloat16()
    layer.forward(x, logits, save=True)
    want = [t.clone() for t in (*layer.backward(dout), layer.gu, layer.gu_s, layer.hg, layer.dgu, layer.dxg)]

    def shifted(t):
        n = 16 // t.element_size()
        return torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")[n:].view(t.shape)

    for name in ("gu", "hg", "dgu", "dxg", "dyg"):
        setattr(layer, name, shifted(getattr(layer, name)))
    layer.forward(x, logits, save=True)
    got = (*layer.backward(dout, shifted(layer.w13), shifted(layer.w2)), layer.gu, layer.gu_s, layer.hg, layer.dgu, layer.dxg)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,H,I,E,K,shared,layout", [(1, 4096, 2048, 8, 2, 1, "masked"), (700, 1152, 5504, 3, 2, 0, "contig"),
                                                     (1500, 2048, 1024, 70, 8, 1, "contig"), (400, 7168, 384, 2, 1, 0, "masked"),
                                                     (64, 128, 128, 1000, 2, 1, "contig"), (5, 128, 128, 1023, 3, 1, "masked")])
def test_larger_sizes(T, H, I, E, K, shared, layout):
    """Several waves of tiles, many slots, long reductions; every stage against 64 bits on the device, by norm.  The
    roundings of operands and results add up in squares: half a step of bf16 is 2^-8 of a value at most, a third of that
    in the mean square; three such stages stay below one half step."""
    layer, r = make_layer(T, H, I, E, K, shared, layout)
    x, logits, dout = r(T, H).bfloat16(), r(T, E), r(T, H).bfloat16()
    layer.forward(x, logits, save=True)
    dx, dlogits, dw13, dw2 = layer.backward(dout)
    torch.cuda.synchronize()
    assert int(layer.err) == 0
    n = E + shared
    m, offs = layer.masked_m.tolist(), layer.offsets.tolist()
    values = torch.empty(layer.rows, 2 * I, device="cuda")
    moe.moe_fp8_dequantize(layer.gu, layer.gu_s, values)
    dxg = torch.zeros(layer.rows, H, dtype=torch.float64, device="cuda")
    worst = {}
    for s in range(n):
        a = s * layer.p.M_max if layout == "masked" else offs[s]
        rows = slice(a, a + m[s])
        if not m[s]:
            assert not dw13[s].any() and not dw2[s].any()
            continue
        xr, wg = layer.xg[rows].double(), layer.wg[rows].double()[:, None]
        gu = xr @ layer.w13[s].double().T
        err = (values[rows].double() - gu).abs()
        # an E4M3 step, and the scale's share of one below the smallest normal number
        sc = layer.gu_s[rows].double().repeat_interleave(128, 1)
        assert (err <= 2.0 ** -4 * gu.abs() * (1 + 2.0 ** -10) + 2.0 ** -9 * sc).all()
        leaf = values[rows].double().requires_grad_()
        h = tref.swiglu(leaf[:, :I], leaf[:, I:])
        dy = layer.dyg[rows].double()
        dgu, = torch.autograd.grad(h, leaf, wg * (dy @ layer.w2[s].double()))
        h = (wg * h).detach()
        dxg[rows] = dgu @ layer.w13[s].double()
        for name, got, want in (("hg", layer.hg[rows], h), ("dgu", layer.dgu[rows], dgu), ("dw13", dw13[s], dgu.T @ xr),
                                ("dw2", dw2[s], dy.T @ h)):
            worst[name] = max(worst.get(name, 0.0), float((got.double() - want).norm() / want.norm()))
    live = torch.zeros(layer.rows, dtype=torch.bool, device="cuda")
    live[layer.row_of.long().flatten()] = True
    worst["dxg"] = float((layer.dxg[live].double() - dxg[live]).norm() / dxg[live].norm())
    want = dxg[layer.row_of.long()].sum(1)
    worst["dx"] = float((dx.double() - want).norm() / want.norm())
    assert max(worst.values()) <= HALF, worst


def test_elements_past_32_bits():
    """Grouped rows whose elements pass 2^31: the last rows of the last slot and the first of the first."""
    T, H, I, E, K = 40000, 128, 14336, 4, 2
    layer, r = make_layer(T, H, I, E, K)
    assert layer.dgu.numel() > 1 << 31
    x, logits, dout = r(T, H).bfloat16(), r(T, E), r(T, H).bfloat16()
    layer.forward(x, logits, save=True)
    dx, dlogits, dw13, dw2 = layer.backward(dout)
    torch.cuda.synchronize()
    assert int(layer.err) == 0
    rows = layer.rows
    for s, part in ((0, slice(0, 40)), (E - 1, slice(rows - 40, rows))):
        xr, wg, dy = layer.xg[part].double(), layer.wg[part].double()[:, None], layer.dyg[part].double()
        gu = xr @ layer.w13[s].double().T
        values = torch.empty(40, 2 * I, device="cuda")
        moe.moe_fp8_dequantize(layer.gu[part], layer.gu_s[part], values)
        sc = layer.gu_s[part].double().repeat_interleave(128, 1)
        assert ((values.double() - gu).abs() <= 2.0 ** -4 * gu.abs() * (1 + 2.0 ** -10) + 2.0 ** -9 * sc).all()
        leaf = values.double().requires_grad_()
        h = tref.swiglu(leaf[:, :I], leaf[:, I:])
        dgu, = torch.autograd.grad(h, leaf, wg * (dy @ layer.w2[s].double()))
        for got, want in ((layer.hg[part], (wg * h).detach()), (layer.dgu[part], dgu),
                          (layer.dxg[part], dgu @ layer.w13[s].double())):
            assert float((got.double() - want).norm() / want.norm()) <= HALF
    # the last slot's gradients of weights, whose rows lie past 2^31 elements, from what the products were given
    n = int(layer.masked_m[-1])
    tail = slice(rows - n, rows)
    for got, a, b in ((dw13[-1][:256], layer.dgu[tail][:, :256], layer.xg[tail]), (dw2[-1], layer.dyg[tail], layer.hg[tail])):
        want = a.double().T @ b.double()
        assert float((got.double() - want).norm() / want.norm()) <= HALF
