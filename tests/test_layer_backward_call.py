"""moe_layer_backward as a program with buffers of its own calls it: every argument in its place, and what it refuses."""
import pytest
import torch

import routed_expert_layer_moe_gb300 as moe

NAMES = ("dout yg row_of ids w xg w13 w2 gu gu_scales masked_m offsets dyg wg dgu hg dxg dw dx dlogits dw13 dw2 "
         "err_flag").split()


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_layer_moe_gb300 import build
    build.build()


def test_refusals():
    """Each argument is looked at under its own name, before anything is launched."""
    p = moe.Problem.make(T=4, H=256, I=128, E=8, K=2, layout="contig")
    none = dict.fromkeys(NAMES)
    with pytest.raises(moe.MoeError):
        moe.moe_layer_backward(p, **none, stream=0)
    host = torch.zeros(4, 256, dtype=torch.bfloat16)
    for name in NAMES:
        with pytest.raises(ValueError, match="expected a CUDA tensor" if name == "err_flag" else name + ":"):
            moe.moe_layer_backward(p, **{**none, name: host}, stream=0)
    for name in ("logits", "add"):
        with pytest.raises(ValueError, match=name + ":"):
            moe.moe_layer_backward(p, **none, **{name: host}, stream=0)
    with pytest.raises(KeyError):
        moe.moe_layer_backward(p, **none, score="argmax", stream=0)
    with pytest.raises(moe.MoeError):
        moe.moe_layer_backward(moe.Problem.make(T=4, H=256, I=128, E=8, K=2, wt="mxfp4"), **none, stream=0)


@pytest.mark.gpu
@pytest.mark.parametrize("score,scale", [("softmax", 1.0), ("sigmoid", 2.5)])
@pytest.mark.parametrize("layout", ["masked", "contig"])
@pytest.mark.parametrize("how", ["bf16", "fp32, added to", "no weights"])
def test_gives_what_the_layer_gives(score, scale, layout, how):
    from test_gpu_train import make_layer
    T, H, I, E, K = 37, 256, 128, 6, 2
    layer, r = make_layer(T, H, I, E, K, 1, layout)
    x, dout, logits, add = r(T, H).bfloat16(), r(T, H).bfloat16(), r(T, E), r(T, E)
    if score == "sigmoid":
        layer.route_grouped(logits, 2, 1, None, True, scale)
        layer.permute(x)
        layer.ffn_save()
    else:
        layer.forward(x, logits, save=True)
    route = dict(score=score, logits=logits, renormalize=True, scale=scale, add=add)
    grads, start = {}, {}
    if how == "fp32, added to":
        start = {"dw13": r(*layer.w13.shape), "dw2": r(*layer.w2.shape)}
        grads = {k: v.clone() for k, v in start.items()}
    want = layer.backward(dout, **grads, accumulate=bool(grads), weights=how != "no weights", **route)
    kept = {k: getattr(layer, k).clone() for k in ("hg", "dgu", "dxg", "dyg", "wg", "dw")}

    def empty(t):
        return torch.full_like(t, 7)

    out = {k: empty(v) for k, v in kept.items()}
    out["dx"], out["dlogits"] = empty(want[0]), empty(want[1])
    if how == "no weights":
        out["dw13"] = out["dw2"] = None
    elif start:
        out.update({k: v.clone() for k, v in start.items()})
    else:
        out["dw13"], out["dw2"] = empty(want[2]), empty(want[3])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.moe_layer_backward(layer.p, dout, layer.yg, layer.row_of, layer.ids, layer.w, layer.xg, layer.w13, layer.w2,
                           layer.gu, layer.gu_s, layer.masked_m, layer.offsets, *(out[k] for k in NAMES[12:22]), err,
                           accumulate=bool(start), **route)
    torch.cuda.synchronize()
    assert int(err) == 0
    for name, v in zip(("dx", "dlogits", "dw13", "dw2"), want):
        assert (v is None and out[name] is None) or torch.equal(out[name], v), name
    live = layer.row_of.flatten().long()
    for name, v in kept.items():
        a, b = (out[name], v) if name == "dw" else (out[name][live], v[live])
        assert torch.equal(a, b), name
    rest = torch.ones(layer.rows, dtype=torch.bool, device="cuda")
    rest[live] = False
    for name in ("hg", "dgu", "dxg", "dyg", "wg"):
        assert (out[name][rest] == 7).all(), name
