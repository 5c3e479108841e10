"""How far an 8-bit checkpoint may be from what it was made of, from the largest numbers of fp32 to the smallest.

With s = amax c + e and c = fp32(1/448), which is a little above 1/448: a quotient x / s of at most 448 becomes a code
within half a step, 2^-4 of it and 2^-10 below 2^-6.  Larger ones saturate; there x - 448 s <= amax (1 - 448 c) - 448 e <=
448 |e|.  |e| <= 2^-24 s for a normal s, which is far within 2^-4; a subnormal one has |e| <= 2^-150, so 448 |e| is up
to 7 * 2^-144, whatever s is."""
import numpy as np
import pytest
import torch

import train_reference as ref

BELOW = 7 * 2.0 ** -144


def groups(dtype):
    """Groups of 128 values whose largest magnitude goes through fp32's exponents, and through the subnormal ones in steps
    that are no powers of two."""
    g = np.random.default_rng(1)
    tops = [m * 2.0 ** e for e in (*range(-149, -120), *range(-120, 128, 9), 127) for m in (1.0, 1.17, 1.34, 1.61, 1.9999999)]
    tops += [k * 2.0 ** -149 for k in (*range(1, 2000, 13), 223, 224, 600, 671, 672)] + [float(np.finfo(np.float32).max)]
    x = np.array(tops)[:, None] * np.concatenate([g.uniform(-1, 1, (len(tops), 64)), 2.0 ** g.uniform(-20, 0, (len(tops), 64))], 1)
    x[:, 17] = tops
    with np.errstate(over="ignore"):
        x = torch.from_numpy(x).float().to(dtype).double()
    return x[torch.isfinite(x).all(1)]


def bound(x, s):
    s = s.double()[:, None].expand(x.shape)
    std = torch.where(x.abs() >= 2.0 ** -6 * s, 2.0 ** -4 * x.abs(), 2.0 ** -10 * s)
    return std + torch.where(s < 2.0 ** -126, BELOW, 0.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_definition(dtype):
    x = groups(dtype)
    codes, scales = ref.fp8_quantize(x.numpy())
    s = torch.from_numpy(scales)[:, 0]
    off = (torch.from_numpy(ref.fp8_values(codes, scales)) - x).abs()
    assert (off <= bound(x, s)).all()
    # The room below the normal scales is needed, and nowhere else.  Not for bf16, whose least magnitude is 2^-133: there
    # 448 |e| is within 2^-8 of the largest one, which a code within half a step has room for.
    tight = (off > bound(x, s) - torch.where(s < 2.0 ** -126, BELOW, 0.0)[:, None]).any(1)
    assert bool(tight.any()) == (dtype is torch.float32) and (s[tight] < 2.0 ** -126).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [128, 130])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_calls(dtype, cols):
    import routed_expert_layer_moe_gb300 as moe
    from routed_expert_layer_moe_gb300 import build
    build.build()
    x = groups(dtype)
    rows = len(x)
    wide = torch.zeros(rows, cols).to(dtype)
    wide[:, :128] = x.to(dtype)
    codes = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, -(-cols // 128), device="cuda")
    out = torch.empty(rows, cols, device="cuda")
    moe.moe_fp8_quantize(wide.cuda(), codes, scales)
    moe.moe_fp8_dequantize(codes, scales, out)
    off = (out[:, :128].cpu().double() - x).abs()
    # and the result's own rounding to fp32
    assert (off <= bound(x, scales[:, 0].cpu()) + 2.0 ** -24 * 1.0625 * x.abs() + 2.0 ** -149).all()
