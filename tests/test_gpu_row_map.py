"""Readers of row_of: an entry outside the grouped buffers is a record without a place, as -1 is."""
import pytest
import torch

import routed_expert_layer_moe_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_layer_moe_gb300 import build
    build.build()
    torch.cuda.init()


def with_strays(row_of, rows):
    """row_of with some records unplaced, and the same with entries outside [0, rows) in their place."""
    none, stray = row_of.clone(), row_of.clone()
    flat = stray.view(-1)
    bad = torch.tensor([rows, rows + 1, 2 ** 31 - 1, -2, -2 ** 31], dtype=torch.int32, device=flat.device)
    at = torch.arange(0, flat.numel(), 3, device=flat.device)
    flat[at] = bad[torch.arange(len(at), device=flat.device) % len(bad)]
    none.view(-1)[at] = -1
    return none, stray


@pytest.mark.parametrize("T,K,shared", [(1, 1, 0), (6, 2, 1), (50, 3, 0)])
@pytest.mark.parametrize("layout", ["masked", "contig"])
def test_gradient(T, K, shared, layout):
    H, I, E = 256, 128, 5
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    p = moe.Problem.make(T=T, H=H, I=I, E=E, K=K, has_shared=shared, M_max=T if layout == "masked" else 0, layout=layout)
    n = E + shared
    layer = moe.MoeLayer(p, "bf16", "bf16", "bf16", (r(n, 2 * I, H) * H ** -0.5).bfloat16(),
                         (r(n, H, I) * I ** -0.5).bfloat16(), train=True)
    layer.forward(r(T, H).bfloat16(), r(T, E), save=True)
    dout = r(T, H).bfloat16()
    dxg = r(layer.rows, H)
    got = []
    for row_of in with_strays(layer.row_of, layer.rows):
        layer.row_of.copy_(row_of)
        for t in (layer.dyg, layer.wg, layer.dxg):
            t.zero_()
        grads = layer.backward(dout)
        dw, wg = torch.empty_like(layer.w), torch.zeros_like(layer.wg)
        dyg, dx = torch.zeros_like(layer.yg), torch.empty_like(layer.out)
        moe.moe_combine_backward(p, dout, layer.yg, row_of, layer.w, dyg, wg, dw)
        moe.moe_permute_backward(p, dxg, row_of, dx)
        out = torch.empty_like(layer.out)
        moe.moe_combine(p, layer.yg, row_of, layer.w, out)
        torch.cuda.synchronize()
        got.append([t.clone() for t in (*grads, layer.dw, dw, wg, dyg, dx, out)])
        assert int(layer.err) == 0
        # the unplaced records have no gradient of their weight
        assert not dw[(row_of[:, :K] < 0) | (row_of[:, :K] >= layer.rows)].any()
        parts = torch.where(((row_of >= 0) & (row_of < layer.rows))[..., None],
                            dxg[row_of.clamp(0, layer.rows - 1).long()].double(), 0.0)
        want = parts.sum(1)
        # a sum of K + S terms in fp32, rounded to bf16
        assert ((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + (K + 1) * 2.0 ** -23 * parts.abs().sum(1)).all()
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("wt", ["f32", "bf16", "mxfp4"])
@pytest.mark.parametrize("T,H,I", [(3, 1024, 2048), (40, 256, 384)])
def test_forward(wt, T, H, I):
    """moe_combine and moe_ffn_combine: decode-sized down products, whose K split ends in the combine, and others."""
    E, K = 4, 2
    f32 = wt == "f32"
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    act = "f32" if f32 else "bf16"
    p = moe.Problem.make(T=T, H=H, I=I, E=E, K=K, act=act, wt=wt, out=act, layout="contig")
    w = [(r(E, 2 * I, H) * H ** -0.5), (r(E, H, I) * I ** -0.5)]
    scales = ()
    if wt == "mxfp4":
        codes = [torch.empty(*t.shape[:-1], t.shape[-1] // 2, dtype=torch.uint8, device="cuda") for t in w]
        scales = [torch.empty(*t.shape[:-1], t.shape[-1] // 32, dtype=torch.uint8, device="cuda") for t in w]
        for t, c, s in zip(w, codes, scales):
            moe.moe_mx_quantize(t, c, s)
        w = codes
    elif not f32:
        w = [t.bfloat16() for t in w]
    layer = moe.MoeLayer(p, act, wt, act, *w, *scales)
    layer.forward(r(T, H).to(layer.out.dtype), r(T, E))
    got = []
    for row_of in with_strays(layer.row_of, layer.rows):
        layer.row_of.copy_(row_of)
        layer.combine()
        plain = layer.out.clone()
        layer.ffn_combine()
        torch.cuda.synchronize()
        assert int(layer.err) == 0
        assert torch.isfinite(plain).all()
        # every record of a token unplaced: zeros
        lost = ((row_of < 0) | (row_of >= layer.rows)).all(1)
        assert not plain[lost].any() and not layer.out[lost].any()
        got.append([plain, layer.out.clone()])
    assert all(torch.equal(a, b) for a, b in zip(*got))
