"""One transformer block's MoE half on MXFP4 experts: weights quantised on load, a decode step captured in a CUDA
graph, and the router's balance loss with its gradient.

    python examples/mxfp4_block.py [tokens]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import routed_expert_layer_moe_gb300 as moe  # noqa: E402


def quantize(w):
    """[experts, rows, cols] weights -> (codes, scales), an expert at a time."""
    n, rows, cols = w.shape
    codes = torch.empty(n, rows, cols // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(n, rows, cols // 32, dtype=torch.uint8, device=w.device)
    for e in range(n):
        moe.moe_mx_quantize(w[e], codes[e], scales[e])
    return codes, scales


def make_block(T, H, I, E, K, device="cuda", seed=0):
    """A block of random weights and its router's matrix."""
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g, device=device) * std + mean  # noqa: E731
    w13, w13_s = quantize(r(E, 2 * I, H, std=0.02))
    w2, w2_s = quantize(r(E, H, I, std=0.02))
    p = moe.Problem.make(T=T, H=H, I=I, E=E, K=K, M_max=T, wt="mxfp4")
    layer = moe.MoeLayer(p, "bf16", "mxfp4", "bf16", w13, w2, w13_s, w2_s, device=device)
    norm = lambda: r(H, std=0.1, mean=1.0).bfloat16()  # noqa: E731
    gate = r(H, std=0.05, mean=0.3).bfloat16()
    return moe.MoeBlock(layer, norm(), norm(), gate, norm()), r(H, E, std=H ** -0.5)


def step(block, w_g, x):
    """Norm, router, layer, norm: the block's output, the next block's normed input, the router's logits."""
    logits = block.enter(x).float() @ w_g
    y, xn = block.leave(x, logits)
    return y, xn, logits


def main():
    T = int(sys.argv[1]) if len(sys.argv) > 1 else 32
    block, w_g = make_block(T, H=1024, I=2048, E=16, K=4)
    x = torch.randn(T, 1024, device="cuda").bfloat16()
    step(block, w_g, x)  # a first eager pass: device attributes are looked up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, xn, logits = step(block, w_g, x)
    graph.replay()
    loss = block.balance(logits)
    dlogits = block.balance_backward(logits, torch.ones_like(loss))
    torch.cuda.synchronize()
    assert int(block.layer.err) == 0
    print("y %s  |y| %.3f  next |xn| %.3f  balance loss %.5f  |dlogits| %.3g  tokens per expert %s" % (
        tuple(y.shape), y.float().norm(), xn.float().norm(), loss.item(), dlogits.norm(), block.counts[0].tolist()))


if __name__ == "__main__":
    main()
