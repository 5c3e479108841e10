"""Plain 64-bit forms of the 8-bit checkpoints and of the gradients that train the experts, on the CPU."""
import numpy as np
import torch

GROUP = 128
# the magnitudes of E4M3 by code (0 .. 0x7E)
MAGNITUDES = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def fp8_codes(q):
    """Codes of the quotients q (64 bits), by nearest distance, ties to the even code, saturating."""
    q = np.asarray(q, np.float64)
    m = np.minimum(np.abs(q), 448.0)
    hi = np.searchsorted(MAGNITUDES, m).clip(1, 126)
    lo = hi - 1
    down, up = m - MAGNITUDES[lo], MAGNITUDES[hi] - m
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return (code + 128 * np.signbit(q)).astype(np.uint8)


def fp8_quantize(x):
    """Codes and fp32 scales of x [rows, cols] (values of fp32 or fewer bits)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    n = -(-cols // GROUP)
    codes, scales = np.zeros(x.shape, np.uint8), np.ones((rows, n), np.float32)
    for g in range(n):
        b = x[:, g * GROUP:(g + 1) * GROUP]
        with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
            s = np.abs(b).max(1).astype(np.float32) * (np.float32(1) / np.float32(448))
        s[s == 0] = 1
        bad = ~np.isfinite(b).all(1)
        s[bad] = np.nan
        q = np.where(bad[:, None], 0.0, b / np.where(bad, 1.0, s.astype(np.float64))[:, None])
        codes[:, g * GROUP:(g + 1) * GROUP] = fp8_codes(q)
        scales[:, g] = s
    return codes, scales


def fp8_values(codes, scales):
    """The values of codes [rows, cols] and scales, in 64 bits."""
    codes, scales = np.asarray(codes), np.asarray(scales, np.float64)
    one = np.concatenate([MAGNITUDES, [np.nan], -MAGNITUDES, [np.nan]])
    return one[codes] * np.repeat(scales, GROUP, 1)[:, :codes.shape[1]]


def swiglu(g, u):
    return g * torch.sigmoid(g) * u


def swiglu_grads(g, u, dh):
    """Gradients of swiglu by automatic differentiation."""
    g, u = g.clone().requires_grad_(), u.clone().requires_grad_()
    return torch.autograd.grad(swiglu(g, u), (g, u), dh)


def route_weights(logits, ids, score, renormalize, scale):
    """The router's weights of the chosen experts, as a function of all logits."""
    l = torch.gather(logits, 1, ids.long())
    if score == "softmax":
        return torch.softmax(l, 1)
    s = torch.sigmoid(l)
    return scale * (s / s.sum(1, keepdim=True) if renormalize else s)
