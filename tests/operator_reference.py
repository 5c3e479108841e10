"""Plain 64-bit forms of the MXFP4, balance-loss and block-norm operators, on the CPU."""
import numpy as np
import torch

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_quantize(x):
    """Codes (one per element) and scale bytes of x [..., n], n a multiple of 32, by nearest distance."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    codes = np.zeros(b.shape, np.uint8)
    scales = np.zeros(b.shape[:-1], np.uint8)
    for i in np.ndindex(*b.shape[:-1]):
        v = b[i]
        if not np.isfinite(v).all():
            scales[i] = 255
            continue
        top = np.abs(v).max()
        e = 0 if top == 0 else int(np.clip(np.frexp(top)[1] - 1 - 2, -127, 125))
        scales[i] = e + 127
        m = np.abs(v) / 2.0 ** e
        d = np.abs(m[:, None] - MAGNITUDES)  # nearest magnitude; of two equally near, the even code
        d = np.where(d == d.min(1, keepdims=True), np.arange(8) % 2, 9)
        codes[i] = d.argmin(1) + 8 * np.signbit(v)
    return codes.reshape(x.shape), scales


def mx_pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def mx_values(packed, scales):
    """The values of packed codes and scale bytes, in 64 bits."""
    packed, scales = np.asarray(packed), np.asarray(scales)
    one = np.concatenate([MAGNITUDES, -MAGNITUDES])
    v = np.stack([one[packed & 15], one[packed >> 4]], -1).reshape(*packed.shape[:-1], -1, 32)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(*packed.shape[:-1], -1)


def random_mx(rng, *shape, std=1.0):
    """Packed codes and scales of random rows, without the (slow) quantiser: random codes, scales of
    the exponents that N(0, std) values have."""
    packed = rng.integers(0, 256, shape[:-1] + (shape[-1] // 2,), dtype=np.uint8)
    e = np.floor(np.log2(std * 2.5 * np.exp(0.3 * rng.standard_normal(shape[:-1] + (shape[-1] // 32,))))) - 2
    return packed, (e + 127).astype(np.uint8)


def balance(logits, ids, valid, seq, score, coef, dloss):
    """Loss, counts, score sums, token counts, and the gradient by automatic differentiation."""
    T, E = logits.shape
    K = ids.shape[1]
    seq = [0, T] if seq is None else [int(v) for v in seq]
    B = len(seq) - 1
    out = dict(loss=torch.zeros(B, dtype=torch.float64), counts=torch.zeros(B, E, dtype=torch.int64),
               prob_sum=torch.zeros(B, E, dtype=torch.float64), tokens=torch.zeros(B, dtype=torch.int64),
               dlogits=torch.zeros(T, E, dtype=torch.float64))
    for b in range(B):
        rows = [t for t in range(seq[b], seq[b + 1]) if valid is None or valid[t]]
        n = len(rows)
        if not n:
            continue
        l = logits[rows].double()
        empty = torch.isinf(l).all(1) & (l < 0).all(1)  # every expert switched off
        l = torch.where(empty[:, None], torch.zeros_like(l), l).requires_grad_()
        p = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
        p = p / p.sum(1, keepdim=True) * (~empty)[:, None]
        for t in rows:
            for k in range(K):
                if 0 <= int(ids[t, k]) < E:
                    out["counts"][b, int(ids[t, k])] += 1
        c = out["counts"][b].double()
        scale = coef * E / (K * n * n)
        # the scores of a token sum to one: counts less their mean have the same gradient, without the rounding of
        # a difference of equal numbers
        (scale * ((c - c.mean()) * p.sum(0)).sum() * float(dloss[b])).backward()
        out["loss"][b] = scale * (c * p.detach().sum(0)).sum()
        out["prob_sum"][b] = p.detach().sum(0)
        out["tokens"][b] = n
        out["dlogits"][rows] = torch.where(torch.isnan(l.grad), torch.zeros_like(l.grad), l.grad)
    return out


def block_norm(x, block, gate, w_post, w_pre, res_scale, eps):
    def rms(v):
        return v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + eps)

    y = x
    if block is not None:
        branch = rms(block) * w_post
        y = x + res_scale * (branch if gate is None else gate * branch)
    return y, None if w_pre is None else rms(y) * w_pre


def block_norm_grads(args, res_scale, eps, dy, dxn):
    """Gradients of x, block, gate, w_post, w_pre (None where there is none)."""
    leaf = [None if a is None else a.double().requires_grad_() for a in args]
    y, xn = block_norm(*leaf, res_scale, eps)
    outs, grads = [], []
    for o, g in ((y, dy), (xn, dxn)):
        if g is not None:
            outs.append(o)
            grads.append(g.double())
    torch.autograd.backward(outs, grads)
    return [None if a is None else (torch.zeros_like(a) if a.grad is None else a.grad) for a in leaf]
