"""backward() answers for a pass that was kept, and for no other."""
import pytest
import torch

import routed_expert_layer_moe_gb300 as moe
from test_gpu_train import make_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_layer_moe_gb300 import build
    build.build()
    torch.cuda.init()


def test_passes_in_turn():
    T, H, E = 40, 256, 5
    layer, r = make_layer(T, H, 128, E, 2, 1)
    block = moe.MoeBlock(layer, r(H).bfloat16(), r(H).bfloat16())
    x, other, dout = (r(T, H).bfloat16() for _ in range(3))
    logits, other_logits = r(T, E), r(T, E)
    with pytest.raises(ValueError, match="save"):
        layer.backward(dout)
    layer.forward(x, logits, save=True)
    want = layer.backward(dout)
    for infer in (lambda: layer.forward(other, other_logits), lambda: layer.forward(other, other_logits, fused=True),
                  lambda: (block.enter(other), block.leave(other, other_logits))):
        infer()
        with pytest.raises(ValueError, match="save"):
            layer.backward(dout)
        layer.forward(x, logits, save=True)
        assert all(torch.equal(a, b) for a, b in zip(layer.backward(dout), want))
    # a pass that keeps g and u when they are wanted
    layer.forward(x, logits)
    yg = layer.yg.clone()
    layer.swiglu_save()
    got = layer.backward(dout)
    layer.forward(x, logits, save=True)
    same_yg = torch.equal(layer.yg, yg)  # its h comes from another kernel, whose sums may round otherwise
    assert all(torch.equal(a, b) for a, b in zip((got[0], *got[2:]), (want[0], *want[2:])))
    assert not same_yg or torch.equal(got[1], want[1])
    assert int(layer.err) == 0


def test_replayed_passes():
    """A captured pass is replayed behind an inference pass: the program says that it was saved."""
    T, H, E = 24, 256, 4
    layer, r = make_layer(T, H, 128, E, 2)
    x, other, dout = (r(T, H).bfloat16() for _ in range(3))
    logits, other_logits = r(T, E), r(T, E)
    layer.forward(x, logits, save=True)
    want = layer.backward(dout)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, logits, save=True)
    layer.forward(other, other_logits)
    graph.replay()
    with pytest.raises(ValueError, match="saved"):
        layer.backward(dout)
    layer.saved = True
    assert all(torch.equal(a, b) for a, b in zip(layer.backward(dout), want))


def test_scratch_in_common():
    """Two layers in flight that have the gradient's scratch in common give what they give with their own."""
    T, H, E = 90, 256, 6
    a, r = make_layer(T, H, 128, E, 2, 1)
    b = moe.MoeLayer(a.p, "bf16", "bf16", "bf16", a.w13, a.w2, train=True)
    data = [(r(T, H).bfloat16(), r(T, E), r(T, H).bfloat16()) for _ in range(2)]
    want = []
    for layer, (x, logits, dout) in zip((a, b), data):
        layer.forward(x, logits, save=True)
        want.append(layer.backward(dout))
    for name in ("dyg", "wg", "dgu", "dxg", "dw"):
        setattr(b, name, getattr(a, name).fill_(float("nan")))
    for layer, (x, logits, _) in zip((a, b), data):
        layer.forward(x, logits, save=True)
    for layer, (_, _, dout), v in list(zip((a, b), data, want))[::-1]:
        assert all(torch.equal(p, q) for p, q in zip(layer.backward(dout), v))
    assert int(a.err) == int(b.err) == 0
