"""Which pass a layer's backward() answers for: the steps' record on the host, with calls that launch nothing."""
import contextlib

import pytest
import torch

import routed_expert_layer_moe_gb300 as moe
from routed_expert_layer_moe_gb300 import layer as layer_module

CALLS = ["moe_route_topk", "moe_route_grouped_topk", "moe_permute", "moe_route_permute", "moe_grouped_swiglu_gemm",
         "moe_grouped_swiglu_gemm_save", "moe_grouped_down_gemm", "moe_grouped_ffn", "moe_combine", "moe_ffn_combine",
         "_layer_backward"]


@pytest.fixture
def make(monkeypatch):
    from routed_expert_layer_moe_gb300 import build
    build.build()
    made = []
    for name in CALLS:
        monkeypatch.setattr(layer_module.L, name, lambda *a, _name=name, **k: made.append(_name))
    monkeypatch.setattr(layer_module.L, "_ptr", lambda t: 0)

    def layer(T=4, train=True):
        p = moe.Problem.make(T=T, H=128, I=128, E=2, K=1, layout="contig")
        w13, w2 = torch.zeros(2, 256, 128, dtype=torch.bfloat16), torch.zeros(2, 128, 128, dtype=torch.bfloat16)
        return moe.MoeLayer(p, "bf16", "bf16", "bf16", w13, w2, device="cpu", train=train)

    layer.made = made
    return layer


PARTS = {  # steps that are no kept pass of their own
    "forward": lambda m: m.forward(None, None), "forward fused": lambda m: m.forward(None, None, fused=True),
    "route": lambda m: m.route(None), "route_grouped": lambda m: m.route_grouped(None, 1, 1),
    "permute": lambda m: m.permute(None), "route_permute": lambda m: m.route_permute(None, None),
    "without down": lambda m: (m.route_permute(None, None), m.swiglu_save()),
    "without g and u": lambda m: (m.permute(None), m.swiglu(), m.down()),
    "g and u of other rows": lambda m: (m.swiglu_save(), m.permute(None), m.ffn()),
    "h of other rows": lambda m: (m.swiglu(), m.permute(None), m.down()),
}
AGAIN = {  # steps that compute the same values of the same rows once more
    "ffn": lambda m: m.ffn(), "ffn_combine": lambda m: m.ffn_combine(), "swiglu": lambda m: m.swiglu(),
    "swiglu and down": lambda m: (m.swiglu(), m.down()), "swiglu_save": lambda m: m.swiglu_save(),
    "down": lambda m: m.down(), "combine": lambda m: m.combine(), "backward": lambda m: m.backward(m.out),
}


def refused(m, made):
    del made[:]
    with pytest.raises(ValueError, match="save"):
        m.backward(m.out)
    return not made


def test_fresh_layer(make):
    assert refused(make(), make.made)


@pytest.mark.parametrize("part", PARTS)
def test_parts_of_a_pass(make, part):
    m = make()
    PARTS[part](m)
    assert refused(m, make.made)
    m.forward(None, None, save=True)
    m.backward(m.out)
    PARTS[part](m)
    assert refused(m, make.made)
    m.forward(None, None, save=True)  # and back again
    m.backward(m.out)
    assert make.made[-1] == "_layer_backward"


@pytest.mark.parametrize("again", AGAIN)
def test_the_same_rows_again(make, again):
    m = make()
    m.forward(None, None, save=True)
    AGAIN[again](m)
    m.backward(m.out)
    assert make.made[-1] == "_layer_backward"


@pytest.mark.parametrize("steps", [
    lambda m: m.forward(None, None, save=True), lambda m: m.forward(None, None, fused=True, save=True),
    lambda m: (m.route_grouped(None, 1, 1), m.permute(None), m.ffn_save()),
    lambda m: (m.route(None), m.permute(None), m.swiglu_save(), m.down(), m.combine()),
    lambda m: (m.forward(None, None), m.swiglu_save()),  # g and u of a pass computed when they are wanted
    lambda m: (m.forward(None, None, fused=True), m.swiglu_save()),
    lambda m: (m.forward(None, None), m.forward(None, None, save=True))])
def test_a_pass_that_was_kept(make, steps):
    m = make()
    steps(m)
    m.backward(m.out)
    assert make.made[-1] == "_layer_backward"


def test_down_after_the_gradient(make):
    """backward() leaves h times its weights in hg: a down() on that is no output of the pass."""
    m = make()
    m.forward(None, None, save=True)
    m.backward(m.out)
    m.down()
    assert refused(m, make.made)
    m.swiglu()
    m.down()
    m.backward(m.out)


def test_failed_call(make, monkeypatch):
    m = make()
    m.forward(None, None, save=True)

    def fails(*a):
        raise moe.MoeError(moe.MOE_ERR_CUDA, "moe_grouped_down_gemm")
    with monkeypatch.context() as c:
        c.setattr(layer_module.L, "moe_grouped_down_gemm", fails)
        with contextlib.suppress(moe.MoeError):
            m.forward(None, None, save=True)
    assert refused(m, make.made)


def test_empty_batch(make):
    m = make(T=0)
    assert refused(m, make.made)
    m.forward(None, None, save=True)
    m.backward(m.out)


def test_replayed_pass(make):
    """Replays of a captured graph make no calls: a program that replays a pass that saves says so."""
    m = make()
    m.forward(None, None, save=True)
    assert m.saved
    m.forward(None, None)
    assert not m.saved
    m.saved = True
    m.backward(m.out)
    m.saved = False
    assert refused(m, make.made)


def test_a_checkpoint_of_the_programs_own(make):
    """Buffers that a program fills itself, in any order."""
    for names in (("ids", "xg", "gu", "gu_s", "yg"), ("gu_s", "yg", "gu", "ids")):
        m = make()
        for name in names:
            setattr(m, name, torch.zeros_like(getattr(m, name)))
        m.backward(m.out)
        assert make.made[-1] == "_layer_backward"
        m.forward(None, None)
        assert refused(m, make.made)


def test_layers_that_are_not_trained(make):
    m = make(train=False)
    m.forward(None, None)
    m.forward(None, None, fused=True)
    m.down()
    assert not m.saved
    with pytest.raises(ValueError, match="train=True"):
        m.backward(m.out)
