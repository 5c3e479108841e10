"""The training pass of a block under a balance loss that counts: every gradient, with the balance loss's own share of it
large enough to be seen.

The reference is the block in 64 bits with the routing's choice held and with the gradient of the experts taken where the
checkpoint has them: products with W2 have the value of the exact h and the gradient of that of the kept g and u, which
pass their own gradients straight through.  Between the inputs and any gradient lie at most ten roundings to bf16, of
2^-8 each at most: xn, h, yg, out, dout, dgu, w h, the layer's dx, dxn and dx."""
import importlib.util
import os

import pytest
import torch

import operator_reference as ref
import train_reference as tref
from test_gpu_train import HALF, d

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOL = 10 * HALF
COEF = 0.01


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


def gradients(block, w_g, x, dy, dxn, dloss, counts=None):
    """Gradients in 64 bits, by name ("x": the block's input), of the pass that the block holds.  counts: the experts'
    counts that the balance loss takes, if not those of the pass."""
    p, layer = block.p, block.layer
    w = {"w_pre": block.w_pre, "w_g": w_g, "w13": layer.w13, "w2": layer.w2, "gate": block.gate, "w_post": block.w_post,
         "w_next": block.w_next, "x": x}
    w = {k: d(v).requires_grad_() for k, v in w.items()}
    ids, row_of = layer.ids.cpu(), layer.row_of.cpu().long()
    kept = torch.from_numpy(tref.fp8_values(layer.gu.cpu().numpy(), layer.gu_s.cpu().numpy()))
    xn = ref.block_norm(w["x"], None, None, None, w["w_pre"], 1.0, 1e-6)[1]
    logits = xn @ w["w_g"]
    weight = tref.route_weights(logits, ids, "softmax", True, 1.0)
    out = torch.zeros_like(xn)
    for e in range(p.E):
        t, k = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        gu = xn[t] @ w["w13"][e].T
        st = gu + (kept[row_of[t, k]] - gu).detach()
        y = tref.swiglu(st[:, :p.I], st[:, p.I:]) @ w["w2"][e].T
        y = y + (tref.swiglu(gu[:, :p.I], gu[:, p.I:]) @ w["w2"][e].T - y).detach()
        out = out.index_add(0, t, weight[t, k][:, None] * y)
    y, xn_next = ref.block_norm(w["x"], out, w["gate"], w["w_post"], w["w_next"], 1.0, 1e-6)
    n = torch.bincount(ids.flatten().long(), minlength=p.E).double() if counts is None else counts
    balance = COEF * p.E / (p.K * p.T ** 2) * (n * torch.softmax(logits, 1).sum(0)).sum()
    ((d(dy) * y).sum() + (d(dxn) * xn_next).sum() + dloss * balance).backward()
    return {k: v.grad for k, v in w.items()}


@pytest.mark.parametrize("T,H,I,E,K", [(70, 256, 384, 5, 2), (130, 128, 256, 12, 3)])
def test_block(example, T, H, I, E, K):
    block, w_g = example.make_block(T, H, I, E, K)
    g = torch.Generator().manual_seed(3)
    x, dy, dxn, other = (torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(4))
    # another pass before it: its counts are not this one's
    _, _, logits = example.forward(block, w_g, other)
    block.balance(logits)
    stale = d(block.counts[0])
    _, _, logits = example.forward(block, w_g, x)
    dloss = 1e6
    args = block, w_g, x, dy, dxn
    want, none, turned = (gradients(*args, v) for v in (dloss, 0.0, -dloss))
    old = gradients(*args, dloss, stale)
    got, without = ({"x": r[0], **r[1]} for r in (
        example.backward(block, w_g, x, logits, dy, dxn, torch.tensor([v], device="cuda")) for v in (dloss, 0.0)))
    torch.cuda.synchronize()
    assert int(block.layer.err) == 0
    for name, v in want.items():
        assert off(got[name], v) <= TOL, name
        assert off(without[name], none[name]) <= TOL, name
    # what reaches the router, and so the test's sight, is large; a lost, turned or stale term does not pass
    for name in ("x", "w_pre", "w_g"):
        for wrong in (none, turned):
            assert float((wrong[name] - want[name]).norm() / want[name].norm()) > 4 * TOL, name
    assert float((old["w_g"] - want["w_g"]).norm() / want["w_g"].norm()) > 4 * TOL
    for name in ("w13", "w2", "gate", "w_post", "w_next"):
        assert torch.equal(got[name], without[name]), name


def test_router_share(example):
    """The balance loss's part of the router's weight, on the operands that the kernels had.  Logits are off by (H + 1)
    2^-24 of their terms' magnitudes (13 in the mean here), so a score by 2^-11 of itself at most; the rest is fp32."""
    T, H, E, K = 90, 256, 7, 2
    block, w_g = example.make_block(T, H, 128, E, K)
    x, dy, dxn = (torch.randn(T, H, device="cuda").bfloat16() for _ in range(3))
    _, _, logits = example.forward(block, w_g, x)
    dloss = 1e6
    a, b = (example.backward(block, w_g, x, logits, dy, dxn, torch.tensor([v], device="cuda"))[1]["w_g"] for v in (dloss, 0.0))
    xn = d(block.xn)
    leaf = d(w_g).requires_grad_()
    n = torch.bincount(block.layer.ids.cpu().flatten().long(), minlength=E).double()
    (dloss * COEF * E / (K * T ** 2) * (n * torch.softmax(xn @ leaf, 1).sum(0)).sum()).backward()
    assert off(a.double() - b.double(), leaf.grad) <= 2.0 ** -10
