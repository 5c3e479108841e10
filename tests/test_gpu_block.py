"""The block that runs the norms, the MXFP4 layer and the router's loss together, as examples/mxfp4_block.py does."""
import importlib.util
import os

import pytest
import torch

import operator_reference as ref
import routed_expert_layer_moe_gb300 as moe

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from routed_expert_layer_moe_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("mxfp4_block", os.path.join(ROOT, "examples", "mxfp4_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("T", [1, 33])
def test_block(example, T):
    H, I, E, K = 256, 384, 8, 2
    block, w_g = example.make_block(T, H, I, E, K)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).bfloat16().cuda()
    y, xn, logits = (t.clone() for t in example.step(block, w_g, x))
    out = block.layer.out.clone()
    torch.cuda.synchronize()
    assert int(block.layer.err) == 0
    d = lambda t: t.double().cpu()  # noqa: E731
    # the norms around the layer's own output, within bf16's rounding (2^-8 allows for a neighbour) and fp32 sums
    want = ref.block_norm(d(x), None, None, None, d(block.w_pre), 1.0, 1e-6)[1]
    assert ((d(block.xn) - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all()
    wy, wxn = ref.block_norm(d(x), d(out), d(block.gate), d(block.w_post), d(block.w_next), 1.0, 1e-6)
    assert ((d(y) - wy).abs() <= 2.0 ** -8 * wy.abs() + 1e-5).all()
    assert ((d(xn) - wxn).abs() <= 2.0 ** -8 * wxn.abs() + 1e-5).all()
    # the layer between them ran on the normed input
    assert torch.equal(block.layer.forward(block.xn, logits), out)
    # the loss of this routing, and its gradient
    dloss = torch.tensor([0.7], device="cuda")
    loss, dl = block.balance(logits), block.balance_backward(logits, dloss)
    r = ref.balance(logits.cpu(), block.layer.ids.cpu(), None, None, "softmax", 0.01, dloss.cpu())
    assert torch.equal(block.counts.cpu().long(), r["counts"]) and int(r["counts"].sum()) == T * K
    assert abs(float(loss) - float(r["loss"][0])) <= 2.0 ** -18 * float(r["loss"][0])
    scale = r["dlogits"].abs().max()
    assert (d(dl) - r["dlogits"]).abs().max() <= 2.0 ** -15 * max(float(scale), 1e-30)
    # gradients of both norms
    dy, dxn = torch.randn_like(y), torch.randn_like(y)
    grads = block.leave_backward(x, dy, dxn)
    want = ref.block_norm_grads([x.cpu(), out.cpu(), block.gate.cpu(), block.w_post.cpu(), block.w_next.cpu()], 1.0, 1e-6,
                                dy.cpu(), dxn.cpu())
    for g, w in zip(grads, want):
        assert (d(g) - w).abs().max() <= 2.0 ** -7 * w.abs().max()
    dx, dw = block.enter_backward(x, dxn, dy)
    want = ref.block_norm_grads([x.cpu(), None, None, None, block.w_pre.cpu()], 1.0, 1e-6, dy.cpu(), dxn.cpu())
    for g, w in ((dx, want[0]), (dw, want[4])):
        assert (d(g) - w).abs().max() <= 2.0 ** -7 * w.abs().max()


def test_block_in_a_graph(example):
    block, w_g = example.make_block(17, 256, 256, 4, 2)
    x = torch.randn(17, 256, device="cuda").bfloat16()
    example.step(block, w_g, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, xn, logits = example.step(block, w_g, x)
        block.balance(logits)
        dl = block.balance_backward(logits, torch.ones(1, device="cuda"))
    x.copy_(torch.randn_like(x))
    graph.replay()
    got = [t.clone() for t in (y, xn, block.loss, dl)]
    y, xn, logits = example.step(block, w_g, x)
    want = [y, xn, block.balance(logits), block.balance_backward(logits, torch.ones(1, device="cuda"))]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def wide_block(T=4096, H=1024, E=64, score="softmax", nseq=1, gate="token"):
    """A block of many tokens and a thin layer, so that its norms and its loss take long enough to overlap."""
    g = torch.Generator(device="cuda").manual_seed(T + E)
    r = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g, device="cuda") * std + mean  # noqa: E731
    q = []
    for s in ((E, 256, H), (E, H, 128)):
        w = r(*s, std=0.05)
        q.append((torch.empty(*s[:2], s[2] // 2, dtype=torch.uint8, device="cuda"),
                  torch.empty(*s[:2], s[2] // 32, dtype=torch.uint8, device="cuda")))
        moe.moe_mx_quantize(w, *q[-1])
    p = moe.Problem.make(T=T, H=H, I=128, E=E, K=4, wt="mxfp4", layout="contig")
    layer = moe.MoeLayer(p, "bf16", "mxfp4", "bf16", q[0][0], q[1][0], q[0][1], q[1][1])
    norm = lambda: r(H, std=0.1, mean=1.0).bfloat16()  # noqa: E731
    gt = {"token": torch.sigmoid(r(T, 1)).bfloat16(), "channel": r(H, std=0.1, mean=0.3).bfloat16(), None: None}[gate]
    return moe.MoeBlock(layer, norm(), norm(), gt, norm(), score=score, nseq=nseq), r


def test_loss_and_norm_gradients_on_their_own_streams(example):
    """balance(), leave_backward() and enter_backward() on three streams at once give what they give in turn."""
    block, r = wide_block()
    T, H, E = block.p.T, block.p.H, block.p.E
    x, logits = r(T, H).bfloat16(), r(T, E)
    dy, dxn = r(T, H).bfloat16(), r(T, H).bfloat16()
    block.enter(x)
    block.leave(x, logits)

    def calls(a=None, b=None, c=None):
        return [block.balance(logits, stream=a), *block.leave_backward(x, dy, dxn, stream=b),
                *block.enter_backward(x, dxn, dy, stream=c)]

    want = [t.clone() for t in calls()]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        torch.cuda.synchronize()
        got = calls(*streams)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_of_a_block_share_no_scratch(example, monkeypatch):
    """balance(), leave_backward() and enter_backward() may run at once on streams of their own."""
    block, r = wide_block(T=40, H=256)
    x, logits, d = r(40, 256).bfloat16(), r(40, 64), r(40, 256).bfloat16()
    block.enter(x)
    block.leave(x, logits)
    spans = []
    from routed_expert_layer_moe_gb300 import _lib

    def recorded(f, at):
        def call(*a):
            spans.append((a[at].data_ptr(), a[at].data_ptr() + a[at].numel()))
            return f(*a)
        return call

    monkeypatch.setattr(_lib, "moe_balance_loss", recorded(_lib.moe_balance_loss, 12))
    monkeypatch.setattr(_lib, "moe_block_norm_backward", recorded(_lib.moe_block_norm_backward, 14))
    block.balance(logits), block.leave_backward(x, d, d), block.enter_backward(x, d)
    assert len(spans) == 3
    spans.sort()
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))


def test_results_belong_to_the_stream_that_writes_them(example):
    """Memory of a dropped result is not handed out on another stream while its kernel may still write it."""
    block, r = wide_block(T=64, H=256)
    x, logits, d = r(64, 256).bfloat16(), r(64, 64), r(64, 256).bfloat16()
    block.enter(x)
    block.leave(x, logits)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for call in (lambda: block.leave_backward(x, d, d, stream=stream), lambda: block.enter_backward(x, d, stream=stream)):
            grads = call()
            sizes = [(g.shape, g.dtype) for g in grads]
            at = {g.data_ptr() for g in grads}
            del grads
            again = [torch.empty(s, dtype=t, device="cuda") for s, t in sizes]
            assert not at & {g.data_ptr() for g in again}
            torch.cuda.synchronize()


def test_gradients_of_an_earlier_pass(example):
    """Two micro-batches forward, then both backward, from what the caller kept of the first."""
    block, r = wide_block(T=300, H=256, score="sigmoid", nseq=2)
    T, H, E = block.p.T, block.p.H, block.p.E
    seq = torch.tensor([0, 120, T], dtype=torch.int32, device="cuda")
    batches = [(r(T, H).bfloat16(), r(T, E), r(T, H).bfloat16(), r(T, H).bfloat16()) for _ in range(2)]
    dloss = torch.tensor([1.0, 0.5], device="cuda")
    want = []
    for x, logits, dy, dxn in batches:  # one after the other
        block.enter(x)
        block.leave(x, logits)
        block.balance(logits, None, seq)
        want.append([t.clone() for t in (block.loss, block.balance_backward(logits, dloss, None, seq),
                                         *block.leave_backward(x, dy, dxn))])
    kept = []
    for x, logits, dy, dxn in batches:
        block.enter(x)
        block.leave(x, logits)
        kept.append((block.layer.out.clone(), block.layer.ids.clone()))
    sums = []
    for (x, logits, dy, dxn), (out, ids) in zip(batches, kept):
        block.balance(logits, None, seq, ids=ids)
        sums.append((block.loss.clone(), block.counts.clone(), block.tokens.clone()))
    for (x, logits, dy, dxn), (out, ids), (loss, counts, tokens), w in zip(batches, kept, sums, want):
        got = [loss, block.balance_backward(logits, dloss, None, seq, counts=counts, tokens=tokens),
               *block.leave_backward(x, dy, dxn, out=out)]
        assert all(torch.equal(a, b) for a, b in zip(got, w))
    with pytest.raises(ValueError, match="belong together"):
        block.balance_backward(logits, dloss, None, seq, counts=counts)


def test_a_routing_of_the_callers_own(example):
    """leave(routed=True) runs the layer on the routing that the layer holds: here the grouped sigmoid router's."""
    block, r = wide_block(T=50, H=256, E=16, score="sigmoid", gate="channel")
    layer, x, logits = block.layer, r(50, 256).bfloat16(), r(50, 16)
    xn = block.enter(x).clone()
    layer.route_grouped(logits, 4, 2, scale=2.5)
    ids, w = layer.ids.clone(), layer.w.clone()
    y, xn_next = (t.clone() for t in block.leave(x, logits, routed=True))
    assert torch.equal(layer.ids, ids) and torch.equal(layer.w, w)
    out = layer.out.clone()
    layer.permute(xn), layer.swiglu(), layer.down(), layer.combine()
    assert torch.equal(layer.out, out) and int(layer.err) == 0
    d = lambda t: t.double().cpu()  # noqa: E731
    wy, wxn = ref.block_norm(d(x), d(out), d(block.gate), d(block.w_post), d(block.w_next), 1.0, 1e-6)
    for got, want in ((y, wy), (xn_next, wxn)):
        assert ((d(got) - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all()
    loss = block.balance(logits)
    want = ref.balance(logits.cpu(), ids.cpu(), None, None, "sigmoid", 0.01, torch.ones(1))
    assert torch.equal(block.counts.cpu().long(), want["counts"])
    assert abs(float(loss) - float(want["loss"][0])) <= 2.0 ** -18 * float(want["loss"][0])


@pytest.mark.parametrize("gate", ["token", "channel", None])
def test_block_with_segments_and_masked_tokens(example, gate):
    """Packed sequences with padding: the block's outputs, its loss per segment and the gradients, with each gate."""
    block, r = wide_block(T=70, H=256, E=16, nseq=3, gate=gate)
    T, H, E = 70, 256, 16
    x, logits, dy, dxn = r(T, H).bfloat16(), r(T, E), r(T, H).bfloat16(), r(T, H).bfloat16()
    seq = torch.tensor([4, 4, 40, 66], dtype=torch.int32, device="cuda")
    valid = (r(T) > -1.0).to(torch.uint8)
    dloss = torch.tensor([1.0, 0.5, -2.0], device="cuda")
    block.enter(x)
    y, xn = block.leave(x, logits)
    loss, dl = block.balance(logits, valid, seq), block.balance_backward(logits, dloss, valid, seq)
    want = ref.balance(logits.cpu(), block.layer.ids.cpu(), valid.cpu(), seq.tolist(), "softmax", 0.01, dloss.cpu())
    d = lambda t: t.double().cpu()  # noqa: E731
    assert torch.equal(block.counts.cpu().long(), want["counts"]) and torch.equal(block.tokens.cpu().long(), want["tokens"])
    assert ((d(loss) - want["loss"]).abs() <= 2.0 ** -18 * want["loss"]).all()
    assert (d(dl) - want["dlogits"]).abs().max() <= 2.0 ** -15 * want["dlogits"].abs().max()
    out = block.layer.out
    host = [None if t is None else t.cpu() for t in (x, out, block.gate, block.w_post, block.w_next)]
    wy, wxn = ref.block_norm(*[None if t is None else t.double() for t in host], 1.0, 1e-6)
    for got, w in ((y, wy), (xn, wxn)):
        assert ((d(got) - w).abs() <= 2.0 ** -8 * w.abs() + 1e-5).all()
    for g, w in zip(block.leave_backward(x, dy, dxn), ref.block_norm_grads(host, 1.0, 1e-6, dy.cpu(), dxn.cpu())):
        assert (g is None) == (w is None)
        if g is not None:
            assert (d(g) - w).abs().max() <= 2.0 ** -7 * w.abs().max()
