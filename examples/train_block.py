"""Gradients of a block of bf16 experts: forward with 8-bit checkpoints of the experts' activations, the balance loss, and the
backward pass from the block's output to every weight and to its input.

    python examples/train_block.py

The router's product and the optimiser are the caller's; everything between them runs in the library's kernels."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import routed_expert_layer_moe_gb300 as moe  # noqa: E402


def make_block(T, H, I, E, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g, device="cuda") * std + mean).bfloat16()  # noqa: E731
    p = moe.Problem.make(T=T, H=H, I=I, E=E, K=K, layout="contig")
    layer = moe.MoeLayer(p, "bf16", "bf16", "bf16", r(E, 2 * I, H, std=H ** -0.5), r(E, H, I, std=I ** -0.5), train=True)
    block = moe.MoeBlock(layer, r(H, std=0.1, mean=1.0), r(H, std=0.1, mean=1.0), r(H, std=0.1, mean=0.3),
                         r(H, std=0.1, mean=1.0))
    w_g = torch.randn(H, E, generator=g, device="cuda") * H ** -0.5
    return block, w_g


def forward(block, w_g, x):
    """(y, the next block's normed input, the router's logits)"""
    logits = block.enter(x).float() @ w_g
    y, xn_next = block.leave(x, logits, save=True)
    return y, xn_next, logits


def backward(block, w_g, x, logits, dy, dxn_next, dloss):
    """Gradients of that pass: of x and, by name, of every weight."""
    block.balance(logits)
    dx, dout, dgate, dw_post, dw_next = block.leave_backward(x, dy, dxn_next)
    dxn, dlogits, dw13, dw2 = block.layer.backward(dout, add=block.balance_backward(logits, dloss))
    dw_g = block.xn.float().T @ dlogits
    dxn = (dxn.float() + dlogits @ w_g.T).bfloat16()
    dx, dw_pre = block.enter_backward(x, dxn, dx)
    return dx, {"w_pre": dw_pre, "w_g": dw_g, "w13": dw13, "w2": dw2, "gate": dgate, "w_post": dw_post, "w_next": dw_next}


def main():
    T, H = 512, 1024
    block, w_g = make_block(T, H, 2048, 16, 2)
    x, target = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(T, H, device="cuda")
    for step in range(3):
        y, xn_next, logits = forward(block, w_g, x)
        err = y.float() - target
        dx, grads = backward(block, w_g, x, logits, (2 * err / err.numel()).bfloat16(), torch.zeros_like(xn_next),
                             torch.ones(1, device="cuda"))
        print("step %d: loss %.4f, balance %.4f, |dW13| %.3g" % (step, float(err.square().mean()), float(block.loss),
                                                                float(grads["w13"].float().norm())))
        for w, g in ((block.layer.w13, grads["w13"]), (block.layer.w2, grads["w2"])):
            w.sub_(5.0 * g)


if __name__ == "__main__":
    main()
