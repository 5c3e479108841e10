"""MXFP4 on the GPU: the conversions bit for bit, the grouped products and the whole layer against 64 bits.

Bounds.  Conversions: none, codes and scales are equal.  A product's terms are exact in fp32 (two-bit mantissas and
powers of two), so its error is the fp32 sum's, at most one unit of 2^-23 of the sum of magnitudes per K = 64
step and as much again within a step, and the result's rounding to bf16 (2^-9 of it; 2^-8 allows for both).  h is
rounded to MXFP4 from a value with that error: it lies within E2M1's rounding of the exact h, at the scale that was
stored, and the stored scale is that of the exact maximum moved by at most the error."""
import numpy as np
import pytest
import torch

import operator_reference as ref
import routed_expert_layer_moe_gb300 as moe

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_layer_moe_gb300 import build
    build.build()
    torch.cuda.init()


def quantize(x):
    c = torch.full(x.shape[:-1] + (x.shape[-1] // 2,), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full(x.shape[:-1] + (x.shape[-1] // 32,), 0x5A, dtype=torch.uint8, device="cuda")
    moe.moe_mx_quantize(x, c, s)
    return c, s


def check_conversions(x):
    codes, scales = ref.mx_quantize(x.double().numpy())
    c, s = quantize(x.cuda())
    assert (s.cpu().numpy() == scales).all()
    assert (c.cpu().numpy() == ref.mx_pack(codes)).all()
    want = ref.mx_values(ref.mx_pack(codes), scales)
    for dt in DT.values():
        out = torch.full(x.shape, -7.0, dtype=dt, device="cuda")
        moe.moe_mx_dequantize(c, s, out)
        np.testing.assert_array_equal(out.double().cpu().numpy(), want)  # exact in both types


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (7, 32), (2, 5, 160), (65, 4096), (1, 33 * 32)])
def test_conversions_of_random_rows(shape, dtype):
    g = torch.Generator().manual_seed(1)
    scale = torch.exp2(torch.randint(-30, 30, shape[:-1] + (1,), generator=g).float())
    check_conversions((torch.randn(shape, generator=g) * scale).to(DT[dtype]))


@pytest.mark.parametrize("dtype", list(DT))
def test_conversions_at_the_edges(dtype):
    """Every tie and its neighbours at many scales; zeros of both signs; subnormal, largest and non-finite values."""
    dt = DT[dtype]
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    eps = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -23
    row = torch.cat([ties, ties * (1 + eps), ties * (1 - eps / 2), torch.tensor([6.0, 7.0, 7.96875, 0.0, -0.0])])
    row = torch.cat([row, -row])[:31]
    rows = []
    for e in (-126, -120, -30, -1, 0, 1, 40, 124):
        for top in (4.0, 6.0, 7.96875):
            rows.append(torch.cat([row.clamp(-top, top), torch.tensor([top])]) * 2.0 ** e)
    zero = torch.zeros(32)
    tiny = torch.linspace(-1, 1, 32) * 2.0 ** -126 * 0.9  # a subnormal maximum
    least = zero.clone()
    least[5] = 2.0 ** -133
    big = torch.full((32,), torch.finfo(dt).max)
    big[::2] *= -0.4
    inf, nan, ninf = torch.ones(32), torch.ones(32), torch.ones(32)
    inf[3], nan[31], ninf[0] = float("inf"), float("nan"), float("-inf")
    both = inf.clone()
    both[4] = float("nan")
    rows += [zero, -zero, tiny, least, big, inf, nan, ninf, both]
    check_conversions(torch.stack(rows).to(dt))


def test_dequantize_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)[:, :256]
    scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(16).view(256, 16)
    want = ref.mx_values(codes.numpy(), scales.numpy())
    out = torch.empty(256, 512, dtype=torch.float32, device="cuda")
    moe.moe_mx_dequantize(codes.cuda(), scales.cuda(), out)
    with np.errstate(over="ignore"):
        np.testing.assert_array_equal(out.cpu().numpy(), want.astype(np.float32))


def test_conversions_use_the_given_stream():
    x = torch.randn(64, 4096, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = torch.zeros(64, 2048, dtype=torch.uint8, device="cuda")
    s = torch.zeros(64, 128, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    moe.moe_mx_quantize(x, c, s, stream=side)
    side.synchronize()
    c2, s2 = quantize(x)
    assert torch.equal(c, c2) and torch.equal(s, s2)


# ---- the products ---------------------------------------------------------------------------------


def problem(sizes, H, I, layout, shared=0, M_max=None, T=None):
    """A problem whose slots hold `sizes` rows (the last one the shared expert's when shared)."""
    E = len(sizes) - shared
    T = max(sizes + [1]) if T is None else T
    K = max(1, min(E, -(-sum(sizes[:E]) // T)))
    while T * K + shared * T < sum(sizes):
        T += 1
    return moe.Problem.make(T=T, H=H, I=I, E=E, K=K, M_max=(M_max or T) if layout == "masked" else 0,
                            has_shared=shared, wt="mxfp4", layout=layout)


class Grouped:
    """Random MXFP4 operands in the grouped layout, on the device, with their 64-bit values on the host."""

    def __init__(self, sizes, H, I, layout, shared=0, M_max=None, seed=0, T=None):
        self.p = p = problem(sizes, H, I, layout, shared, M_max, T)
        assert moe.moe_check_problem(p) == moe.MOE_OK
        self.sizes, self.S = sizes, len(sizes)
        rng = np.random.default_rng(seed)
        rows = moe.moe_grouped_rows(p)
        off = np.concatenate([[0], np.cumsum(sizes)])
        self.first = [s * p.M_max if layout == "masked" else off[s] for s in range(self.S)]
        self.rows = rows
        self.w13 = ref.random_mx(rng, self.S, 2 * I, H, std=0.03)
        self.w2 = ref.random_mx(rng, self.S, H, I, std=0.03)
        self.xg = ref.random_mx(rng, rows, H)
        self.hg = ref.random_mx(rng, rows, I)
        cu = lambda a: tuple(torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in a)  # noqa: E731
        self.d13, self.d2, self.dx, self.dh = cu(self.w13), cu(self.w2), cu(self.xg), cu(self.hg)
        self.m = torch.tensor(sizes, dtype=torch.int32, device="cuda")
        self.off = torch.tensor(off, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(moe.moe_workspace_bytes(p), dtype=torch.uint8, device="cuda")

    def valid(self):
        """(slot, first row, rows) of the rows that hold tokens."""
        for s in range(self.S):
            n = min(self.sizes[s], self.p.M_max) if self.p.layout == moe.MOE_LAYOUT_MASKED else self.sizes[s]
            if n:
                yield s, self.first[s], n

    def check_tiles(self, step):
        tile = moe.moe_gemm_tile_rows(self.p, step)
        st = self.ws[:moe.MOE_STATS_BYTES].view(torch.int32).cpu().numpy().reshape(2, moe.MOE_STATS_CTAS, 2)
        assert st[0, :, 1].sum() == sum(-(-n // tile) for _, _, n in self.valid())


def dot_bound(a, w):
    """Largest error of an fp32 sum of exact products (see the head of this file)."""
    K = a.shape[-1]
    return (K / 64 + 1) * 2.0 ** -22 * (np.abs(a) @ np.abs(w).T)


SIZES = [
    ([5, 0, 1, 17], 256, 256, "masked", 0, None),
    ([16, 15, 31, 32, 33, 63, 64, 65], 384, 128, "masked", 0, None),
    ([127, 128, 129, 200, 257], 256, 384, "masked", 0, 257),
    ([127, 0, 129, 200, 1, 257], 640, 256, "contig", 0, None),
    ([3, 9, 12], 128, 640, "masked", 1, None),   # the shared expert, K of half a stage
    ([40, 7, 41], 512, 1024, "contig", 1, None),
    ([1], 128, 128, "masked", 0, None),          # one token, one expert
    ([2, 3], 256, 4096, "masked", 0, None),      # few tiles: the down product is split along K
    ([2, 130], 384, 4480, "contig", 0, None),    # split, with a last stage of half a K step, an odd tile
    ([0, 0], 256, 256, "masked", 0, 4),          # nothing at all
    ([9, 3], 256, 256, "masked", 0, 6),          # a slot whose count is above M_max: M_max rows
    # slots of 128 rows or more on average: SM pairs, chunks of up to 256 rows in two unequal halves
    ([300, 256, 513, 1, 130], 512, 384, "contig", 0, None),
    ([600, 0, 255, 257], 768, 1024, "masked", 0, 600),
    ([700, 3, 700], 256, 640, "contig", 1, None),
    # 144 pairs of 128-row gate/up tiles (fewer take 64-row tiles on 152 SMs)
    ([16, 15, 31, 32, 33, 63, 64, 65, 127, 128, 1, 2, 0, 100, 90, 17], 256, 1152, "masked", 0, 128),
    ([16, 15, 31, 32, 33, 63, 64, 65, 127, 128, 1, 2, 0, 100, 90, 17], 384, 1152, "contig", 0, None),
]


@pytest.mark.parametrize("case", range(len(SIZES)))
def test_down_product(case):
    sizes, H, I, layout, shared, M_max = SIZES[case]
    g = Grouped(sizes, H, I, layout, shared, M_max, seed=case)
    y = torch.full((g.rows, H), -3.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_down_gemm(g.p, g.dh[0], g.dh[1], g.d2[0], g.d2[1], g.m, g.off, y, g.err, g.ws)
    torch.cuda.synchronize()
    assert int(g.err) == 0
    g.check_tiles(4)
    got = y.double().cpu().numpy()
    seen = np.zeros(g.rows, bool)
    for s, r, n in g.valid():
        a, w = ref.mx_values(g.hg[0][r:r + n], g.hg[1][r:r + n]), ref.mx_values(g.w2[0][s], g.w2[1][s])
        want = a @ w.T
        assert (np.abs(got[r:r + n] - want) <= 2.0 ** -8 * np.abs(want) + dot_bound(a, w)).all()
        seen[r:r + n] = True
    assert (got[~seen] == -3.0).all()  # padding rows are not written


def check_h(h, amax_err, want, codes, scales):
    """Stored MXFP4 h against the exact one (see the head of this file)."""
    b = want.reshape(want.shape[0], -1, 32)
    err = amax_err.reshape(b.shape)
    top = np.abs(b).max(-1)
    e = scales.astype(np.int64) - 127
    slack = err.max(-1)
    for t, sign in ((top - slack, 1), (top + slack, -1)):
        lim = np.floor(np.log2(np.maximum(t, 2.0 ** -140))) - 2
        assert (sign * (e - np.clip(lim, -127, 125)) >= 0).all()
    unit = 2.0 ** e[..., None].astype(np.float64)
    m = np.abs(b) / unit
    half = np.where(m < 2, 0.25, np.where(m < 4, 0.5, np.where(m < 6, 1.0, m - 6 + 1e-9)))
    half = np.maximum(half, np.where(m >= 6, m - 6, 0))
    # a value within the error of a binade's edge may take the other binade's step
    edge = np.where((np.abs(m - 2) * unit <= err) | (np.abs(m - 4) * unit <= err), 2.0, 1.0)
    assert (np.abs(h.reshape(b.shape) - b) <= half * edge * unit + err + 1e-300).all()


@pytest.mark.parametrize("case", range(len(SIZES)))
def test_gate_up_product(case):
    sizes, H, I, layout, shared, M_max = SIZES[case]
    g = Grouped(sizes, H, I, layout, shared, M_max, seed=100 + case)
    hq = torch.full((g.rows, I // 2), 0x5A, dtype=torch.uint8, device="cuda")
    hs = torch.full((g.rows, I // 32), 0x5A, dtype=torch.uint8, device="cuda")
    moe.moe_grouped_swiglu_gemm(g.p, g.dx[0], g.dx[1], g.d13[0], g.d13[1], g.m, g.off, hq, hs, g.err, g.ws)
    torch.cuda.synchronize()
    assert int(g.err) == 0
    g.check_tiles(3)
    hq, hs = hq.cpu().numpy(), hs.cpu().numpy()
    seen = np.zeros(g.rows, bool)
    for s, r, n in g.valid():
        a, w = ref.mx_values(g.xg[0][r:r + n], g.xg[1][r:r + n]), ref.mx_values(g.w13[0][s], g.w13[1][s])
        gu, d = a @ w.T, dot_bound(a, w)
        gate, up = gu[:, :I], gu[:, I:]
        sig = 1 / (1 + np.exp(-gate))
        want = gate * sig * up
        # first-order error of SiLU(g) u: its slope is at most 1.1; 2^-19 for the fast exponential and division
        err = 1.1 * d[:, :I] * (np.abs(up) + d[:, I:]) + np.abs(gate * sig) * d[:, I:] + 2.0 ** -19 * np.abs(want)
        check_h(ref.mx_values(hq[r:r + n], hs[r:r + n]), err, want, hq[r:r + n], hs[r:r + n])
        seen[r:r + n] = True
    assert (hq[~seen] == 0x5A).all() and (hs[~seen] == 0x5A).all()


def test_one_hot_products_read_every_scale_and_code():
    """A row with a single non-zero code reads one column of the weights: exact, for every column of a tile and
    every scale of a row, so a misplaced scale or code cannot hide in a sum."""
    H, I, n = 256, 640, 640
    g = Grouped([n], H, I, "contig", seed=5)
    codes = np.zeros((n, I), np.uint8)
    codes[np.arange(n), np.arange(n)] = 2 + 8 * (np.arange(n) % 2)  # +-1
    scales = np.random.default_rng(6).integers(100, 140, (n, I // 32)).astype(np.uint8)
    hq, hs = torch.from_numpy(ref.mx_pack(codes)).cuda(), torch.from_numpy(scales).cuda()
    y = torch.empty(n, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_down_gemm(g.p, hq, hs, g.d2[0], g.d2[1], g.m, g.off, y, g.err, g.ws)
    want = ref.mx_values(ref.mx_pack(codes), scales) @ ref.mx_values(g.w2[0][0], g.w2[1][0]).T
    np.testing.assert_array_equal(y.double().cpu().numpy(), want)


def test_nan_scales_reach_their_rows_only():
    g = Grouped([40, 9], 256, 512, "masked", seed=7)
    g.dh[1][3, 5] = 255
    y = torch.zeros(g.rows, 256, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_down_gemm(g.p, g.dh[0], g.dh[1], g.d2[0], g.d2[1], g.m, g.off, y, g.err, g.ws)
    bad = torch.isnan(y).cpu()
    assert bad[3].all() and not bad[:3].any() and not bad[4:].any()


def test_products_are_deterministic():
    g = Grouped([2, 3], 256, 4096, "masked", seed=8)
    ys = []
    for _ in range(3):
        y = torch.zeros(g.rows, 256, dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_down_gemm(g.p, g.dh[0], g.dh[1], g.d2[0], g.d2[1], g.m, g.off, y, g.err, g.ws)
        ys.append(y)
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


# ---- the layer --------------------------------------------------------------------------------------


def layer_reference(L, x, logits, p2l=None):
    """The layer in 64 bits: quantised x, exact products, h and the weights as their MXFP4 forms."""
    p = L.p
    xq = ref.mx_values(*[np.asarray(v) for v in (lambda c, s: (ref.mx_pack(c), s))(*ref.mx_quantize(x.double().numpy()))])
    values = lambda c, s: ref.mx_values(c.cpu().numpy(), s.cpu().numpy())  # noqa: E731
    w13 = [values(L.w13[s], L.w13_s[s]) for s in range(p.P + p.has_shared)]
    w2 = [values(L.w2[s], L.w2_s[s]) for s in range(p.P + p.has_shared)]

    def expert(s, row):
        gu = row @ w13[s].T
        h = gu[:p.I] / (1 + np.exp(-gu[:p.I])) * gu[p.I:]
        c, sc = ref.mx_quantize(h[None])
        return ref.mx_values(ref.mx_pack(c), sc)[0] @ w2[s].T

    out = np.zeros((p.T, p.H))
    lg = logits.double().numpy()
    for t in range(p.T):
        ids = sorted(range(p.E), key=lambda e: (-lg[t, e], e))[:p.K]
        w = np.exp(lg[t, ids] - lg[t, ids].max())
        w /= w.sum()
        for k, e in enumerate(ids):
            slots = [e] if p2l is None else [s for s in range(p.P) if p2l[s] == e]
            out[t] += w[k] * expert(slots[t % len(slots)], xq[t])
        if p.has_shared:
            out[t] += expert(p.P, xq[t])
    return out


@pytest.mark.parametrize("T,H,I,E,K,shared,layout,extra", [
    (1, 256, 384, 8, 2, 0, "masked", 0), (7, 384, 256, 5, 3, 1, "masked", 0), (40, 256, 256, 8, 4, 1, "contig", 0),
    (33, 256, 128, 6, 2, 0, "masked", 3), (1100, 128, 128, 8, 4, 0, "contig", 0)])
def test_layer(T, H, I, E, K, shared, layout, extra):
    g = torch.Generator().manual_seed(T)
    P = E + extra
    p = moe.Problem.make(T=T, H=H, I=I, E=E, K=K, P=P, M_max=T if layout == "masked" else 0, has_shared=shared,
                         wt="mxfp4", layout=layout)
    p2l = None if not extra else np.array(list(range(E)) + [1, 1, 4][:extra], np.int32)
    x, logits = torch.randn(T, H, generator=g).bfloat16(), torch.randn(T, E, generator=g)
    order = list(range(E)) + ([] if p2l is None else list(p2l[E:])) + ([E] if shared else [])
    w13, w2 = torch.randn(E + shared, 2 * I, H, generator=g) * 0.05, torch.randn(E + shared, H, I, generator=g) * 0.05
    q13, q2 = quantize(w13[order].cuda()), quantize(w2[order].cuda())
    L = moe.MoeLayer(p, "bf16", "mxfp4", "bf16", q13[0], q2[0], q13[1], q2[1],
                     phys_to_log=None if p2l is None else torch.from_numpy(p2l).cuda())
    out = L.forward(x.cuda(), logits.cuda()).clone()
    yg, xg, xs = L.yg.clone(), L.xg.clone(), L.xg_s.clone()
    torch.cuda.synchronize()
    assert int(L.err) == 0
    # dispatched rows: the quantised tokens, bit for bit
    codes, scales = ref.mx_quantize(x.double().numpy())
    row_of = L.row_of.cpu().numpy()
    for k in range(K + shared):
        assert (xg.cpu().numpy()[row_of[:, k]] == ref.mx_pack(codes)).all()
        assert (xs.cpu().numpy()[row_of[:, k]] == scales).all()
    if T <= 64:
        want = layer_reference(L, x, logits, p2l)
        assert np.abs(out.double().cpu().numpy() - want).max() <= 3e-2 * np.abs(want).max()
    # the fused calls: the same bits
    assert torch.equal(L.forward(x.cuda(), logits.cuda(), fused=True), out)
    rows = torch.from_numpy(np.unique(row_of)).cuda().long()
    assert torch.equal(L.yg[rows], yg[rows])
    L.route(logits.cuda()), L.permute(x.cuda()), L.ffn(), L.combine()
    assert torch.equal(L.out, out)


def test_layer_in_a_graph():
    T, H, I, E, K = 6, 256, 256, 4, 2
    p = moe.Problem.make(T=T, H=H, I=I, E=E, K=K, M_max=T, wt="mxfp4")
    g = torch.Generator().manual_seed(3)
    q13, q2 = (quantize((torch.randn(E, *s, generator=g) * 0.05).cuda()) for s in ((2 * I, H), (H, I)))
    L = moe.MoeLayer(p, "bf16", "mxfp4", "bf16", q13[0], q2[0], q13[1], q2[1])
    x, logits = torch.randn(T, H, generator=g).bfloat16().cuda(), torch.randn(T, E, generator=g).cuda()
    L.forward(x, logits, fused=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.forward(x, logits, fused=True)
    x2, lg2 = torch.randn(T, H, generator=g).bfloat16().cuda(), torch.randn(T, E, generator=g).cuda()
    want = L.forward(x2, lg2).clone()
    x.copy_(x2), logits.copy_(lg2)
    L.out.zero_()
    graph.replay()
    assert torch.equal(L.out, want)


def test_overflowing_h_marks_its_blocks():
    """Columns of h that are infinite or NaN give their blocks of 32 the scale byte 255 and codes 0, the others keep theirs;
    single CTAs with tiles of 64 and of 128 weight rows, and SM pairs."""
    for sizes, I in (([9, 3], 256), ([16, 15, 31, 32, 33, 63, 64, 65, 127, 128, 1, 2, 0, 100, 90, 17], 1152),
                     ([300, 256, 513, 1, 130], 384)):
        H = 256
        g = Grouped(sizes, H, I, "contig", seed=I)

        def h():
            hq = torch.full((g.rows, I // 2), 0x5A, dtype=torch.uint8, device="cuda")
            hs = torch.full((g.rows, I // 32), 0x5A, dtype=torch.uint8, device="cuda")
            moe.moe_grouped_swiglu_gemm(g.p, g.dx[0], g.dx[1], g.d13[0], g.d13[1], g.m, g.off, hq, hs, g.err, g.ws)
            return hq, hs

        hq, hs = h()
        bad = [1, I // 32 - 2]  # blocks of 32 columns
        g.d13[1][:, 40] = 255                     # a NaN in a row of W1
        g.d13[1][:, I + I - 40] = 254             # a row of W3 whose products with x pass the largest fp32
        g.d13[0][:, I + I - 40] = 0x77            # all 6
        first = next(g.valid())[1]
        g.dx[0][first] = 0x77
        g.dx[1][first] = 160                      # x = 6 * 2^33: certainly infinite
        want_q, want_s = hq.clone(), hs.clone()
        hq, hs = h()
        torch.cuda.synchronize()
        assert int(g.err) == 0
        for s, r, n in g.valid():
            rows = slice(r, r + n)
            assert (hs[rows, 1] == 255).all() and (hq[rows, 16:32] == 0).all()
        assert int(hs[first, bad[1]]) == 255 and (hq[first, 16 * bad[1]:16 * bad[1] + 16] == 0).all()
        keep = [b for b in range(I // 32) if b not in bad]
        others = torch.tensor([r for s, a, n in g.valid() for r in range(a, a + n) if r != first], device="cuda")
        cols = torch.tensor([16 * b + i for b in keep for i in range(16)], device="cuda")
        keep = torch.tensor(keep, device="cuda")
        assert torch.equal(hs[others][:, keep], want_s[others][:, keep])
        assert torch.equal(hq[others][:, cols], want_q[others][:, cols])


def random_layer(T, H, I, E, K, layout, seed):
    g = torch.Generator().manual_seed(seed)
    p = moe.Problem.make(T=T, H=H, I=I, E=E, K=K, M_max=T if layout == "masked" else 0, wt="mxfp4", layout=layout)
    q13, q2 = (quantize((torch.randn(E, *s, generator=g) * 0.05).cuda()) for s in ((2 * I, H), (H, I)))
    L = moe.MoeLayer(p, "bf16", "mxfp4", "bf16", q13[0], q2[0], q13[1], q2[1])
    return L, torch.randn(T, H, generator=g).bfloat16(), torch.randn(T, E, generator=g)


@pytest.mark.parametrize("T,H,I,E,K,layout", [
    (3, 256, 384, 8, 2, "masked"), (40, 256, 256, 8, 4, "contig"), (600, 512, 256, 4, 2, "contig"),
    (1100, 256, 128, 8, 4, "masked")])
def test_non_finite_tokens_stay_in_their_rows(T, H, I, E, K, layout):
    """A NaN or an infinity in a token makes its own output NaN and no other token's."""
    L, x, logits = random_layer(T, H, I, E, K, layout, T)
    want = L.forward(x.cuda(), logits.cuda(), fused=True).clone()
    bad = [0, T // 2, T - 1]
    for t, (c, v) in zip(bad, ((5, float("nan")), (H - 1, float("inf")), (H // 2, -float("inf")))):
        x[t, c] = v
    for fused in (True, False):
        out = L.forward(x.cuda(), logits.cuda(), fused=fused)
        torch.cuda.synchronize()
        assert int(L.err) == 0
        assert torch.isnan(out[bad]).all()
        rest = torch.ones(T, dtype=torch.bool)
        rest[bad] = False
        assert torch.equal(out[rest.cuda()], want[rest.cuda()])


@pytest.mark.parametrize("T,H,I,E,K,layout", [(600, 512, 256, 4, 2, "contig"), (1100, 256, 128, 8, 4, "masked"),
                                              (1030, 256, 256, 16, 3, "contig")])
def test_layer_of_prefill_size(T, H, I, E, K, layout):
    """The whole layer on SM pairs against 64 bits, 48 of its tokens.  h is stored in four bits: next
    to a tie its code may be the neighbour of the exact one's, a relative error of up to 1/2 in one of I terms, so the
    bound on an output is 3e-2 of the largest, as in test_layer."""
    L, x, logits = random_layer(T, H, I, E, K, layout, T + 1)
    out = L.forward(x.cuda(), logits.cuda(), fused=True).double().cpu().numpy()
    assert int(L.err) == 0
    tokens = np.random.default_rng(T).choice(T, 48, replace=False)
    sub = moe.Problem.make(T=48, H=H, I=I, E=E, K=K, M_max=48, wt="mxfp4")
    want = layer_reference(type("S", (), dict(p=sub, w13=L.w13, w13_s=L.w13_s, w2=L.w2, w2_s=L.w2_s)), x[tokens],
                           logits[tokens])
    assert np.abs(out[tokens] - want).max() <= 3e-2 * np.abs(want).max()
