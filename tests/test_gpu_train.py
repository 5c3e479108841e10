"""What trains the experts, against 64 bits: the gate/up product that keeps its results in 8 bits, the gradients of
the experts, of the combine, of the dispatch and of the router.

Bounds.  A product of n terms on the tensor cores: sixteen terms at a time are added to an fp32 sum, each step off by at
most 2^-22 of the terms' magnitudes (the sum's rounding or truncation, 2^-23, and the sixteen products' alignment to the
largest, 2^-23), so (n / 16 + 2) 2^-22 of sum |a b| in all.  bf16 results add 2^-8 of themselves.  The elementary
functions of SwiGLU in fp32 are within 2^-18 of the magnitudes that they are made of (the exponential within 2^-21 times
its argument, |g| <= 8 here).  Each stage is compared on the operands that it was given, the roundings of the stage
before it among them."""
import numpy as np
import pytest
import torch

import routed_expert_layer_moe_gb300 as moe
import train_reference as ref

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8  # half a step of bf16, relative
ROWS = 77         # a sentinel for rows that no call writes


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_layer_moe_gb300 import build
    build.build()
    torch.cuda.init()


def sums(n):
    return (n / 16 + 2) * 2.0 ** -22


class Case:
    """A problem with given row counts: grouped inputs on the device, padding rows full of NaN."""

    def __init__(self, counts, H, I, layout, seed=0, slack=3):
        g = torch.Generator().manual_seed(seed + H + I + len(counts))
        self.r = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
        self.counts, self.H, self.I = counts, H, I
        E, R = len(counts), sum(counts)
        M = max(counts) + slack
        T = max(R, 1) if layout == "contig" else M
        self.p = moe.Problem.make(T=T, H=H, I=I, E=E, K=1, M_max=M if layout == "masked" else 0, layout=layout)
        self.rows = moe.moe_grouped_rows(self.p)
        starts = np.concatenate([[0], np.cumsum(counts)])
        base = [e * M for e in range(E)] if layout == "masked" else starts[:-1]
        self.slot = [slice(int(b), int(b) + c) for b, c in zip(base, counts)]
        self.live = torch.zeros(self.rows, dtype=torch.bool)
        for s in self.slot:
            self.live[s] = True
        self.masked_m = torch.tensor(counts, dtype=torch.int32).cuda()
        self.offsets = torch.tensor(starts, dtype=torch.int32).cuda()
        self.err = torch.zeros(1, dtype=torch.int32).cuda()
        self.w13 = self.r(E, 2 * I, H, std=1.0 / H ** 0.5).bfloat16()
        self.w2 = self.r(E, H, I, std=1.0 / I ** 0.5).bfloat16()
        self.x, self.dyg = self.grouped(H), self.grouped(H)

    def grouped(self, cols, std=1.0):
        v = self.r(self.rows, cols, std=std).bfloat16()
        v[~self.live] = float("nan")
        return v

    def out(self, cols, dtype=torch.bfloat16):
        return torch.full((self.rows, cols), ROWS, dtype=dtype, device="cuda")

    def untouched(self, *bufs):
        return all((b.cpu()[~self.live] == ROWS).all() for b in bufs)

    def checkpoint(self):
        codes, scales = ref.fp8_quantize(self.r(self.rows, 2 * self.I, std=1.5).numpy())
        codes, scales = torch.from_numpy(codes), torch.from_numpy(scales)
        scales[~self.live] = float("nan")
        self.wg = torch.rand(self.rows, generator=torch.Generator().manual_seed(self.rows)) * 1.5
        self.wg[~self.live] = float("nan")
        return codes, scales

    def save(self, xg=None):
        hg, gu = self.out(self.I), self.out(2 * self.I, torch.uint8)
        gs = self.out(2 * self.I // 128, torch.float32)
        moe.moe_grouped_swiglu_gemm_save(self.p, (self.x if xg is None else xg).cuda(), self.w13.cuda(), self.masked_m,
                                         self.offsets, hg, gu, gs, self.err)
        torch.cuda.synchronize()
        assert int(self.err) == 0
        return hg, gu, gs

    def backward(self, gu, gs, dtype=torch.bfloat16, dw=None, accumulate=False, dyg=None, xg=None, want=(1, 1, 1)):
        E, H, I = len(self.counts), self.H, self.I
        dgu, hg, dxg = self.out(2 * I), self.out(I), self.out(H, torch.float32)
        dw13, dw2 = dw or (torch.full((E, 2 * I, H), 5.0, dtype=dtype, device="cuda"),
                           torch.full((E, H, I), 5.0, dtype=dtype, device="cuda"))
        a = [t if k else None for k, t in zip(want, (dxg, dw13, dw2))]
        moe.moe_grouped_ffn_backward(self.p, (self.dyg if dyg is None else dyg).cuda(), self.wg.cuda(),
                                     (self.x if xg is None else xg).cuda(), self.w13.cuda(), self.w2.cuda(), gu.cuda(),
                                     gs.cuda(), self.masked_m, self.offsets, dgu, hg, *a, self.err, accumulate)
        torch.cuda.synchronize()
        assert int(self.err) == 0
        return dgu, hg, dxg, dw13, dw2


# counts that leave slots empty, with one row, with 16s and around them, several chunks of 256, ragged everywhere
COUNTS = [[5], [1, 0, 2], [0, 16, 17, 15, 0], [64, 63, 65, 1], [128, 300, 0, 31, 257], [600, 7]]
SIZES = [(128, 128), (256, 384), (640, 128), (384, 1152)]


def d(t):
    return t.cpu().double()


@pytest.mark.parametrize("layout", ["masked", "contig"])
@pytest.mark.parametrize("H,I", SIZES)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_swiglu_save(counts, H, I, layout):
    c = Case(counts, H, I, layout)
    hg, gu, gs = c.save()
    assert c.untouched(hg, gu, gs)
    for e, s in enumerate(c.slot):
        if not c.counts[e]:
            continue
        x, w = d(c.x[s]), d(c.w13[e])
        full, off = x @ w.T, sums(H) * (x.abs() @ w.abs().T)  # g and u, and how far the kernel's may be
        g, u, dg, du = full[:, :I], full[:, I:], off[:, :I], off[:, I:]
        h = ref.swiglu(g, u)
        # the slope of silu is within 1.1, silu within |g|
        bound = HALF * h.abs() + (1 + HALF) * (1.1 * dg * (u.abs() + du) + g.abs() * du + 2.0 ** -18 * (g * u).abs())
        assert ((d(hg[s]) - h).abs() <= bound).all()
        sc = d(gs[s])
        top = full.view(-1, 2 * I // 128, 128).abs().amax(-1)
        doff = off.view(-1, 2 * I // 128, 128).amax(-1)
        assert ((sc - top / 448).abs() <= doff / 448 + 2.0 ** -22 * top / 448).all()  # two roundings of 2^-24, and room
        # rounding is monotone: the code stands for a value between those of both ends of what the kernel's quotient
        # may be (the reciprocal of the scale and the product with it: 2^-22 of the quotient)
        sr = sc.repeat_interleave(128, 1)
        q, dq = full / sr, off / sr + 2.0 ** -22 * (full / sr).abs()
        one = torch.ones_like(sc)
        lo, hi, got = (ref.fp8_values(v, one) for v in (ref.fp8_codes((q - dq).numpy()), ref.fp8_codes((q + dq).numpy()),
                                                        gu[s].cpu().numpy()))
        assert ((lo <= got) & (got <= hi)).all()


@pytest.mark.parametrize("layout", ["masked", "contig"])
@pytest.mark.parametrize("H,I", SIZES)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_ffn_backward(counts, H, I, layout, dtype):
    c = Case(counts, H, I, layout)
    gu, gs = c.checkpoint()
    dgu, hg, dxg, dw13, dw2 = c.backward(gu, gs, dtype)
    assert c.untouched(dgu, hg, dxg)
    values = torch.from_numpy(ref.fp8_values(gu.numpy(), gs.numpy()))
    w_half = HALF if dtype is torch.bfloat16 else 2.0 ** -24
    for e, s in enumerate(c.slot):
        if not c.counts[e]:
            assert not dw13[e].any() and not dw2[e].any()
            continue
        dy, x, w13, w2 = d(c.dyg[s]), d(c.x[s]), d(c.w13[e]), d(c.w2[e])
        g, u = values[s][:, :I], values[s][:, I:]
        w = d(c.wg[s])[:, None]
        h = w * ref.swiglu(g, u)
        assert ((d(hg[s]) - h).abs() <= HALF * h.abs() + 2.0 ** -17 * (w * g * u).abs()).all()
        dh, off = w * (dy @ w2), sums(H) * w * (dy.abs() @ w2.abs())
        want = ref.swiglu_grads(g, u, dh)
        for got, v, k in ((dgu[s][:, :I], want[0], u.abs() * (1 + g.abs())), (dgu[s][:, I:], want[1], g.abs())):
            assert ((d(got) - v).abs() <= HALF * v.abs() + (1 + HALF) * k * (off + 2.0 ** -17 * dh.abs())).all()
        da, hh, n = d(dgu[s]), d(hg[s]), c.counts[e]
        for got, a, b, k, half in ((dxg[s], da, w13, 2 * I, 2.0 ** -24), (dw13[e], da.T, x, n, w_half),
                                   (dw2[e], dy.T, hh, n, w_half)):
            v = a @ b
            assert ((d(got) - v).abs() <= half * v.abs() + (1 + half) * sums(k) * (a.abs() @ b.abs())).all()


@pytest.mark.parametrize("layout", ["masked", "contig"])
def test_differences(layout):
    """dgu and hg against differences of the function itself, in 64 bits: L(g, u) = sum of w dyg (W2 h(g, u))."""
    c = Case([3, 0, 18], 128, 128, layout)
    gu, gs = c.checkpoint()
    dgu = d(c.backward(gu, gs)[0])
    values = torch.from_numpy(ref.fp8_values(gu.numpy(), gs.numpy()))
    I, step = c.I, 1e-5
    for e, s in enumerate(c.slot):
        dy, w2, w = d(c.dyg[s]), d(c.w2[e]), d(c.wg[s])[:, None]

        def loss(gu_):
            return (w * dy * (ref.swiglu(gu_[:, :I], gu_[:, I:]) @ w2.T)).sum(1)  # by row: a row's depends on its own

        for col in range(0, 2 * I, 37):
            a, b = values[s].clone(), values[s].clone()
            a[:, col] += step
            b[:, col] -= step
            slope = (loss(a) - loss(b)) / (2 * step)
            g, u = values[s][:, col % I], values[s][:, I + col % I]
            k = u.abs() * (1 + g.abs()) if col < I else g.abs()
            off = (sums(c.H) + 2.0 ** -17) * (w * (dy.abs() @ w2.abs()))[:, col % I]
            # the differences' own error: third derivatives of size |u dh|, times the step squared, and rounding
            tiny = 1e-8 * (1 + (w * (dy.abs() @ w2.abs()))[:, col % I] * (1 + u.abs()))
            assert ((dgu[s][:, col] - slope).abs() <= HALF * slope.abs() + (1 + HALF) * k * off + tiny).all()


@pytest.mark.parametrize("layout", ["masked", "contig"])
def test_a_slot_with_nan_stays_its_own(layout):
    """NaN in one slot's rows reaches no other slot's results, though tiles read across the border."""
    c = Case([21, 40, 9], 256, 128, layout)
    gu, gs = c.checkpoint()
    clean = c.backward(gu, gs)
    hg, g8, g8s = c.save()
    x, dyg = c.x.clone(), c.dyg.clone()
    x[c.slot[1]] = float("nan")
    dyg[c.slot[1]] = float("inf")
    bad = c.backward(gu, gs, dyg=dyg, xg=x)
    hb, b8, b8s = c.save(x)
    for e in (0, 2):
        for a, b in zip((*clean[:3], hg, g8, g8s), (*bad[:3], hb, b8, b8s)):
            assert torch.equal(a[c.slot[e]], b[c.slot[e]])
        assert torch.equal(clean[3][e], bad[3][e]) and torch.equal(clean[4][e], bad[4][e])
    assert torch.isnan(b8s[c.slot[1]]).all() and not b8[c.slot[1]].any() and torch.isnan(hb[c.slot[1]]).all()
    assert torch.isnan(bad[3][1]).any()


def test_accumulate_and_parts():
    c = Case([33, 0, 100], 256, 384, "contig")
    gu, gs = c.checkpoint()
    dgu, hg, dxg, dw13, dw2 = c.backward(gu, gs, torch.float32)
    start = [torch.randn_like(dw13), torch.randn_like(dw2)]
    got = c.backward(gu, gs, torch.float32, dw=tuple(t.clone() for t in start), accumulate=True)
    assert torch.equal(got[3], start[0] + dw13) and torch.equal(got[4], start[1] + dw2)
    assert torch.equal(got[0], dgu) and torch.equal(got[1], hg) and torch.equal(got[2], dxg)
    for want in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 0, 0)):
        part = c.backward(gu, gs, torch.float32, want=want)
        for k, a, b, left in zip(want, part[2:], (dxg, dw13, dw2), (ROWS, 5.0, 5.0)):
            assert torch.equal(a, b) if k else bool((a == left).all())
        assert torch.equal(part[0], dgu) and torch.equal(part[1], hg)
    c.wg = torch.ones(c.rows)
    one = c.backward(gu, gs)
    E, H, I = 3, c.H, c.I
    out = c.out(2 * I), c.out(I)
    moe.moe_grouped_ffn_backward(c.p, c.dyg.cuda(), None, None, c.w13.cuda(), c.w2.cuda(), gu.cuda(), gs.cuda(),
                                 c.masked_m, c.offsets, *out, None, None, None, c.err)
    assert torch.equal(out[0], one[0]) and torch.equal(out[1], one[1])


def test_no_rows():
    for layout in ("masked", "contig"):
        c = Case([0, 0], 128, 128, layout)
        p = moe.Problem.make(T=0, H=128, I=128, E=2, K=1, M_max=3 if layout == "masked" else 0, layout=layout)
        c.p = p
        c.rows = moe.moe_grouped_rows(p)
        c.live = torch.zeros(c.rows, dtype=torch.bool)
        z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        dw = torch.full((2, 256, 128), 5.0, device="cuda"), torch.full((2, 128, 128), 5.0, device="cuda")
        moe.moe_grouped_ffn_backward(p, z(c.rows, 128), None, z(c.rows, 128), c.w13.cuda(), c.w2.cuda(),
                                     z(c.rows, 256, dt=torch.uint8), z(c.rows, 2, dt=torch.float32), c.masked_m,
                                     c.offsets, z(c.rows, 256), z(c.rows, 128), z(c.rows, 128, dt=torch.float32), *dw, c.err)
        assert not dw[0].any() and not dw[1].any() and int(c.err) == 0
        moe.moe_grouped_swiglu_gemm_save(p, z(c.rows, 128), c.w13.cuda(), c.masked_m, c.offsets, z(c.rows, 128),
                                         z(c.rows, 256, dt=torch.uint8), z(c.rows, 2, dt=torch.float32), c.err)


def test_counts_that_lie_outside_are_cut():
    """Counts and offsets that pass the buffers' ends lead to no access outside them."""
    c = Case([40, 24], 128, 128, "contig")
    gu, gs = c.checkpoint()
    want = c.backward(gu, gs)
    c.masked_m = torch.tensor([40, 9999], dtype=torch.int32, device="cuda")
    got = c.backward(gu, gs)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    c.offsets = torch.tensor([0, -5, 64], dtype=torch.int32, device="cuda")
    got = c.backward(gu, gs)
    assert torch.equal(got[3][0], want[3][0]) and not got[3][1].any()


@pytest.mark.parametrize("T,H,E,K,shared", [(1, 128, 4, 1, 0), (5, 256, 8, 3, 1), (33, 1152, 16, 9, 1), (7, 640, 40, 32, 0),
                                            (300, 128, 4, 2, 0)])
def test_gradients_around_the_experts(T, H, E, K, shared):
    g = torch.Generator().manual_seed(T + H)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = moe.Problem.make(T=T, H=H, I=128, E=E, K=K, has_shared=shared, layout="contig")
    rows = moe.moe_grouped_rows(p)
    row_of = torch.randperm(rows, generator=g)[:T * (K + shared)].view(T, K + shared).int()
    row_of[T // 2, 0] = -1  # a record that was not placed
    dout, yg, w = r(T, H).bfloat16(), r(rows, H).bfloat16(), torch.rand(T, K, generator=g)
    dyg, wg = torch.full((rows, H), 7.0, device="cuda").bfloat16(), torch.full((rows,), 7.0, device="cuda")
    dw = torch.full((T, K), 7.0, device="cuda")
    a = dout.cuda(), yg.cuda(), row_of.cuda(), w.cuda()
    moe.moe_combine_backward(p, *a, dyg, wg, dw)
    left = torch.ones(rows, dtype=torch.bool)
    for t in range(T):
        for k in range(K + shared):
            at = int(row_of[t, k])
            if at < 0:
                assert float(dw[t, k]) == 0
                continue
            left[at] = False
            assert torch.equal(dyg[at].cpu(), dout[t]) and float(wg[at]) == (float(w[t, k]) if k < K else 1.0)
            if k < K:
                prod = dout[t].double() * yg[at].double()
                # a lane's chain of H / 32 products at most and five more sums of 2^-24 each
                assert abs(float(dw[t, k]) - prod.sum()) <= (H / 32 + 5) * 2.0 ** -24 * prod.abs().sum()
    assert (dyg.cpu()[left] == 7).all() and (wg.cpu()[left] == 7).all()
    again = [t.clone() for t in (dyg, wg, dw)]
    inplace = yg.cuda()
    moe.moe_combine_backward(p, a[0], inplace, a[2], a[3], inplace, wg, dw)  # dyg is yg
    assert torch.equal(dw, again[2]) and torch.equal(inplace.cpu()[~left], again[0].cpu()[~left])
    moe.moe_combine_backward(p, a[0], None, a[2], a[3], dyg, wg, None)
    assert torch.equal(dyg, again[0])
    # the dispatch's gradient
    dx = torch.empty(T, H, device="cuda").bfloat16()
    dxg = r(rows, H)
    moe.moe_permute_backward(p, dxg.cuda(), a[2], dx)
    for t in range(T):
        parts = torch.stack([dxg[int(at)].double() if at >= 0 else torch.zeros(H).double() for at in row_of[t]])
        v = parts.sum(0)
        assert ((dx[t].cpu().double() - v).abs() <= HALF * v.abs() + (1 + HALF) * (K + 1) * 2.0 ** -24 * parts.abs().sum(0)).all()


@pytest.mark.parametrize("score,renorm,scale", [("softmax", True, 1.0), ("sigmoid", True, 2.5), ("sigmoid", False, 0.5)])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 8, 2), (130, 257, 32), (9, 1024, 10)])
def test_route_backward(T, E, K, score, renorm, scale):
    g = torch.Generator().manual_seed(E + K)
    logits = torch.randn(T, E, generator=g) * 3
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int()
    dw = torch.randn(T, K, generator=g)
    p = moe.Problem.make(T=T, H=128, I=128, E=E, K=K, layout="contig")
    leaf = logits.double().requires_grad_()
    w = ref.route_weights(leaf, ids, score, renorm, scale)
    (w * dw.double()).sum().backward()
    wf = w.detach().float().cuda()
    out = torch.full((T, E), 7.0, device="cuda")
    args = (logits.cuda(), ids.cuda(), wf, dw.cuda())
    moe.moe_route_backward(p, score, *args, out, renormalize=renorm, scale=scale)
    # weights times a difference of a sum of K terms: 2^-24 for each of K terms and ten operations, expf within 2^-22
    mag = (w.detach() / (1 if score == "softmax" else scale)).abs() * (dw.double().abs() + dw.double().abs().max(1, keepdim=True).values)
    bound = torch.zeros(T, E).double().scatter_(1, ids.long(), max(1.0, scale) * (K + 16) * 2.0 ** -23 * mag)
    assert ((d(out) - leaf.grad).abs() <= bound + 1e-30).all()
    add = torch.randn(T, E, generator=g).cuda()
    both = add.clone()
    moe.moe_route_backward(p, score, args[0] if score == "sigmoid" else None, args[1],
                           args[2] if score == "softmax" else None, args[3], both, both, renorm, scale)
    assert torch.equal(both, add + out)
    # against differences
    if E <= 8:
        for t in range(T):
            for e in range(E):
                hi, lo = logits.double().clone(), logits.double().clone()
                hi[t, e] += 1e-5
                lo[t, e] -= 1e-5
                f = lambda l: (ref.route_weights(l, ids, score, renorm, scale) * dw.double()).sum()  # noqa: E731
                assert abs((f(hi) - f(lo)) / 2e-5 - float(out[t, e])) <= bound[t, e] + 1e-8


def test_route_backward_at_the_edges():
    p = moe.Problem.make(T=4, H=128, I=128, E=4, K=3, layout="contig")
    ids = torch.tensor([[0, 0, 1], [2, 9, -1], [0, 1, 2], [3, 2, 1]], dtype=torch.int32).cuda()
    dw = torch.tensor([[1.0, 2.0, 3.0], [1.0, 5.0, 7.0], [1.0, -1.0, 2.0], [0.0, 0.0, 0.0]]).cuda()
    w = torch.full((4, 3), 0.25).cuda()
    out = torch.empty(4, 4, device="cuda")
    moe.moe_route_backward(p, "softmax", None, ids, w, dw, out)
    # an expert named twice gets both parts; ids outside are skipped
    s = 0.25 * 6
    assert torch.allclose(out[0], torch.tensor([0.25 * (3 - 2 * s), 0.25 * (3 - s), 0, 0]).cuda(), atol=1e-6)
    assert torch.allclose(out[1], torch.tensor([0, 0, 0.25 * (1 - 0.25), 0]).cuda(), atol=1e-6)
    logits = torch.full((4, 4), -200.0).cuda()  # every sigmoid is zero
    logits[3] = 200.0
    moe.moe_route_backward(p, "sigmoid", logits, ids, None, dw, out)
    assert not out.any()


# ---------------------------------------------------------------------------------------------- 8-bit checkpoints

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,offset", [(1, 1, 0), (3, 127, 0), (2, 128, 0), (5, 128, 1), (7, 129, 0), (33, 300, 3), (9, 130, 0), (6, 260, 2), (11, 252, 4),
                                              (2, 4096, 0), (200, 384, 0), (1, 16384, 8)])
def test_fp8_checkpoint(rows, cols, offset, dtype):
    g = torch.Generator().manual_seed(rows * cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(5 * torch.randn(rows, 1, generator=g))
    x.view(-1)[:: 13] = 0.0
    x.view(-1)[5:: 29] = -0.0
    check_fp8(x.to(dtype), offset)


def check_fp8(x, offset=0):
    rows, cols = x.shape
    n = -(-cols // 128)
    place = lambda t: torch.cat([torch.zeros(offset, dtype=t.dtype), t.reshape(-1)]).cuda()[offset:].view(t.shape)  # noqa: E731
    xd, codes = place(x), place(torch.full((rows, cols), 9, dtype=torch.uint8))
    scales, out = torch.full((rows, n), 9.0, device="cuda"), place(torch.full_like(x, 9.0))
    moe.moe_fp8_quantize(xd, codes, scales)
    want_c, want_s = ref.fp8_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    moe.moe_fp8_dequantize(codes, scales, out)
    v = ref.fp8_values(want_c, want_s)
    # code * s in fp32 (exact in 64 bits before it), then the type's own rounding
    want = torch.from_numpy(v).float().to(x.dtype)
    assert torch.equal(out.cpu().nan_to_num(123.0), want.nan_to_num(123.0))
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))


@pytest.mark.parametrize("cols", [128, 130])
def test_fp8_borders(cols):
    """Quotients at the middle between two codes and one step of fp32 to either side, largest and smallest numbers,
    NaN and infinities, groups of zeros."""
    mid = np.concatenate([(ref.MAGNITUDES[1:] + ref.MAGNITUDES[:-1]) / 2, ref.MAGNITUDES]).astype(np.float32)
    rows = []
    for s in (np.float32(1), np.float32(0.7), np.float32(3e-20), np.float32(1.1e-38), np.float32(5e30)):
        v = mid * s
        for w in (v, np.nextafter(v, np.float32(np.inf)), np.nextafter(v, np.float32(0))):
            for i in range(0, len(w), 127):
                row = np.zeros(cols, np.float32)
                part = w[i:i + 127]
                row[:len(part)] = part * np.where(np.arange(len(part)) % 2, -1, 1)
                row[127] = np.float32(448) * s  # the group's largest
                rows.append(row)
    special = np.zeros((8, cols), np.float32)
    special[1, 3], special[2, 7], special[3, 127] = np.nan, np.inf, -np.inf
    special[4] = np.float32(3.4028235e38)
    special[5] = np.float32(1e-45)
    special[6, ::3] = np.float32(-1e-42)
    special[7, -1] = -0.0
    check_fp8(torch.from_numpy(np.concatenate([np.stack(rows), special])))
    check_fp8(torch.from_numpy(special).bfloat16())


# ---------------------------------------------------------------------------------------------- a whole pass

def make_layer(T, H, I, E, K, shared=0, layout="contig", P=None, seed=1, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    P = E if P is None else P
    p = moe.Problem.make(T=T, H=H, I=I, E=E, K=K, P=P, has_shared=shared, M_max=T if layout == "masked" else 0, layout=layout)
    n = P + shared
    w13, w2 = r(n, 2 * I, H, std=H ** -0.5).bfloat16(), r(n, H, I, std=I ** -0.5).bfloat16()
    return moe.MoeLayer(p, "bf16", "bf16", "bf16", w13, w2, train=True, **kw), r


def layer_reference(layer, dout, score="softmax", logits=None, renorm=True, scale=1.0):
    """Gradients of the pass that the layer holds, by automatic differentiation over its own routing and with g and u
    as its checkpoint holds them (their gradients pass straight through the rounding)."""
    p = layer.p
    values = torch.from_numpy(ref.fp8_values(layer.gu.cpu().numpy(), layer.gu_s.cpu().numpy()))
    w13, w2 = d(layer.w13).requires_grad_(), d(layer.w2).requires_grad_()
    l = d(logits).requires_grad_()
    w = ref.route_weights(l, layer.ids.cpu(), score, renorm, scale)
    rows, off = layer.row_of.cpu(), None
    x = {}
    out = torch.zeros(p.T, p.H, dtype=torch.float64)
    # the slot of a grouped row
    m = layer.masked_m.cpu().tolist()
    start = [s * p.M_max for s in range(len(m))] if p.layout == moe.MOE_LAYOUT_MASKED else layer.offsets.cpu().tolist()
    slot = {start[s] + i: s for s in range(len(m)) for i in range(m[s])}
    tokens = d(layer.xg)
    x_leaf = {}
    dlw = torch.zeros(p.T, p.K, dtype=torch.float64)
    yg = d(layer.yg)
    total = 0.0
    for t in range(p.T):
        for k in range(p.K + p.has_shared):
            at = int(rows[t, k])
            if at < 0:
                continue
            s = slot[at]
            xl = x_leaf.setdefault(t, tokens[at].clone().requires_grad_())
            gu = w13[s] @ xl
            gu = gu + (values[at] - gu).detach()
            y = w2[s] @ ref.swiglu(gu[:p.I], gu[p.I:])
            wk = w[t, k].detach() if k < p.K else 1.0
            total = total + (d(dout)[t] * y * wk).sum()
            if k < p.K:  # the combine's own inputs are the rounded yg
                total = total + (w[t, k] - wk) * (d(dout)[t] @ yg[at])
    total.backward()
    dx = torch.stack([x_leaf[t].grad if t in x_leaf else torch.zeros(p.H).double() for t in range(p.T)])
    return dx, l.grad, w13.grad, w2.grad


@pytest.mark.parametrize("T,K,shared,layout", [(1, 1, 0, "contig"), (19, 2, 1, "masked"), (40, 3, 0, "masked"), (23, 2, 1, "contig")])
def test_layer_backward(T, K, shared, layout):
    layer, r = make_layer(T, 256, 384, 5, K, shared, layout)
    x, logits, dout = r(T, 256).bfloat16(), r(T, 5), r(T, 256).bfloat16()
    out = layer.forward(x, logits, save=True).clone()
    plain = moe.MoeLayer(layer.p, "bf16", "bf16", "bf16", layer.w13, layer.w2)
    want = plain.forward(x, logits)
    # the same products summed in another order, rounded to bf16 twice on the way
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -6 * want.float().abs().max()
    grads = layer.backward(dout)
    torch.cuda.synchronize()
    assert int(layer.err) == 0
    # two roundings of operands (dgu; h with w) and those of the results: 4 half steps of the largest magnitudes'
    # accumulated terms; the norm of the error is far below the sum of the terms' bounds
    for got, v, name in zip(grads, layer_reference(layer, dout, logits=logits), ("dx", "dlogits", "dw13", "dw2")):
        rel = float((d(got) - v).norm() / max(float(v.norm()), 1e-30)) if v.abs().max() > 1e-12 else float(d(got).abs().max())
        assert rel <= 4 * HALF, (name, rel)
    again = layer.backward(dout)  # nothing of the pass is used up
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_call_gives_what_the_four_give(score):
    layer, r = make_layer(45, 256, 128, 6, 3, 1)
    x, logits, dout, add = r(45, 256).bfloat16(), r(45, 6), r(45, 256).bfloat16(), r(45, 6)
    how = dict(renormalize=True, scale=2.5)
    if score == "sigmoid":
        layer.route_grouped(logits, 2, 1, None, True, 2.5)
        layer.permute(x)
        layer.ffn_save()
    else:
        layer.forward(x, logits, save=True)
    got = layer.backward(dout, score=score, logits=logits, add=add, **how)
    p = layer.p
    dyg, dgu, hg = (torch.empty_like(t) for t in (layer.yg, layer.dgu, layer.hg))
    wg, dw, dxg = torch.empty_like(layer.wg), torch.empty_like(layer.w), torch.empty_like(layer.dxg)
    dx, dl = torch.empty_like(x), torch.empty_like(logits)
    dw13, dw2 = torch.empty_like(layer.w13), torch.empty_like(layer.w2)
    moe.moe_combine_backward(p, dout, layer.yg, layer.row_of, layer.w, dyg, wg, dw)
    moe.moe_grouped_ffn_backward(p, dyg, wg, layer.xg, layer.w13, layer.w2, layer.gu, layer.gu_s, layer.masked_m,
                                 layer.offsets, dgu, hg, dxg, dw13, dw2, layer.err)
    moe.moe_permute_backward(p, dxg, layer.row_of, dx)
    moe.moe_route_backward(p, score, logits, layer.ids, layer.w, dw, dl, add, **how)
    for a, b in zip(got, (dx, dl, dw13, dw2)):
        assert torch.equal(a, b)
    assert torch.equal(layer.dw, dw) and int(layer.err) == 0
    want = layer_reference(layer, dout, score, logits, **{"renorm": True, "scale": 2.5})
    for a, v in zip((dx, dl - add, dw13, dw2), want):
        assert float((d(a) - v).norm() / v.norm()) <= 4 * HALF


@pytest.mark.parametrize("size", [1e-18, 3e-20, 1e17])
def test_checkpoint_of_tiny_and_huge_products(size):
    """g and u next to the ends of fp32: scales below the smallest normal number, whose reciprocal overflows, and large ones."""
    c = Case([19, 3], 128, 128, "contig")
    c.w13 = (c.w13.double() * size).bfloat16()
    x = (c.x.double() * size).bfloat16()
    hg, gu, gs = c.save(x)
    values = torch.from_numpy(ref.fp8_values(gu.cpu().numpy(), gs.cpu().numpy()))
    for e, s in enumerate(c.slot):
        a, w = d(x[s]), d(c.w13[e])
        g, off = a @ w.T, sums(128) * (a.abs() @ w.abs().T) + 128 * 2.0 ** -126  # products below 2^-126 may be lost
        sc = d(gs[s]).repeat_interleave(128, 1)
        assert torch.isfinite(values[s]).all()
        # half a step of E4M3 (of the smallest binade below it), an off sum, and the scale's own rounding (2^-149 steps)
        assert ((values[s] - g).abs() <= (2.0 ** -4 + 2.0 ** -10) * g.abs() + 2.0 ** -9 * sc + 2 * off + 448 * 2.0 ** -148).all()


@pytest.mark.parametrize("shape", [(5,), (2, 3, 130), (2, 2, 2, 128), (0, 128), (4, 0), (0,)], ids=str)
def test_fp8_shapes(shape):
    """Leading dimensions are rows; nothing is done where there is nothing."""
    x = torch.randn(shape, generator=torch.Generator().manual_seed(1))
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(*shape[:-1], -(-shape[-1] // 128), device="cuda")
    out = torch.empty(shape, device="cuda")
    moe.moe_fp8_quantize(x.cuda(), codes, scales)
    moe.moe_fp8_dequantize(codes, scales, out)
    if x.numel():
        flat = x.reshape(-1, shape[-1])
        c, s = ref.fp8_quantize(flat.double().numpy())
        assert np.array_equal(codes.cpu().numpy().reshape(flat.shape), c)
        assert np.array_equal(scales.cpu().numpy().reshape(s.shape), s)
        assert np.array_equal(out.cpu().numpy().reshape(flat.shape), ref.fp8_values(c, s).astype(np.float32))
    with pytest.raises(ValueError):
        moe.moe_fp8_quantize(x.cuda(), codes, torch.empty(3, 7, 11, device="cuda"))
    if len(shape) > 1 and x.numel():
        with pytest.raises(ValueError, match="dense"):
            moe.moe_fp8_quantize(x.cuda().transpose(0, 1), codes.transpose(0, 1), scales)
