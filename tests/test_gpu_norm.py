"""The norms around the layer, forward and backward, against 64 bits and against differences.

Bounds, relative to the size of what is summed.  fp32 arithmetic with sums over H <= 16384 columns (trees of at
most 2^5 serial adds a thread): 2^-18 of the terms' magnitudes.  A result stored as bf16 adds its rounding, 2^-9 of it
(2^-8 allows for a neighbour).  The sums over T tokens are of fp32 terms in chains of at most T / 300 + 8 adds:
2^-18 of the sum of magnitudes as well."""
import pytest
import torch

import operator_reference as ref
import routed_expert_layer_moe_gb300 as moe

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS, RS = 1e-6, 0.7


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_layer_moe_gb300 import build
    build.build()
    torch.cuda.init()


def inputs(T, H, dtype, gate, block=True, pre=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g) * std + mean).to(DT[dtype])  # noqa: E731
    x, b, wp, wn = r(T, H, std=2.0), r(T, H, std=0.5), r(H, std=0.2, mean=1.0), r(H, std=0.2, mean=1.0)
    gt = {"none": None, "channel": r(H, std=0.3, mean=0.4), "token": r(T, 1, std=0.3, mean=0.4)}[gate]
    if not block:
        b, gt, wp = None, None, None
    return [x, b, gt, wp, wn if pre else None], r(T, H), r(T, H) if pre else None


def dev(t, offset=0):
    if t is None:
        return None
    if not offset:
        return t.cuda()
    buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
    buf[offset:] = t.reshape(-1).cuda()
    return buf[offset:].view(t.shape)


def forward(args, offset=0, stream=None):
    d = [dev(a, offset) for a in args]
    y, xn = (dev(torch.full_like(args[0], -7.0), offset) for _ in range(2))
    torch.cuda.synchronize()
    moe.moe_block_norm(*d, RS, EPS, y, xn if args[4] is not None else None, stream=stream)
    torch.cuda.synchronize()
    return y.cpu(), xn.cpu() if args[4] is not None else None


def backward(args, dy, dxn, offset=0, stream=None):
    x, b, gt, wp, wn = args
    T, H = x.shape
    d = [dev(a, offset) for a in args]
    dyd, dxnd = dev(dy, offset), dev(dxn, offset)
    f = lambda t: None if t is None else torch.full(t.shape, -7.0, device="cuda")  # noqa: E731
    dx, db = dev(torch.full_like(x, -7.0), offset), None if b is None else dev(torch.full_like(x, -7.0), offset)
    dgate, dwp, dwn = f(gt), f(wp), f(wn)
    ws = torch.full((moe.moe_block_norm_workspace_bytes(T, H),), 0xA5, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    moe.moe_block_norm_backward(*d, RS, EPS, dyd, dxnd, dx, db, dgate, dwp, dwn, ws, stream=stream)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu() for t in (dx, db, dgate, dwp, dwn)]


def close(got, want, size, stored):
    """|got - want| within the bounds at the head, `size` the magnitude of the summed terms."""
    d = (got.double() - want).abs()
    lim = 2.0 ** -18 * size + (2.0 ** -8 * want.abs() if stored == torch.bfloat16 else 2.0 ** -22 * want.abs())
    assert (d <= lim + 1e-30).all(), float((d - lim).max())


def check_forward(args, got):
    x, b = args[0], args[1]
    y, xn = ref.block_norm(*[None if a is None else a.double() for a in args], RS, EPS)
    close(got[0], y, x.double().abs() + (y - x.double()).abs(), x.dtype)
    if xn is not None:
        close(got[1], xn, xn.abs() + xn.abs().mean(1, keepdim=True), x.dtype)


def check_backward(args, dy, dxn, got):
    x, b, gt, wp, wn = (None if a is None else a.double() for a in args)
    T, H = x.shape
    dx, db, dgate, dwp, dwn = ref.block_norm_grads(args, RS, EPS, dy, dxn)
    y, _ = ref.block_norm(x, b, gt, wp, wn, RS, EPS)
    ry = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)
    size = torch.zeros_like(x) if dy is None else dy.double().abs()
    if dxn is not None:
        q = dxn.double() * wn
        size = size + ry * (q.abs() + (y * ry).abs() * (q * y * ry).abs().mean(1, keepdim=True))
    close(got[0], dx, size, args[0].dtype)
    if b is not None:
        rb = 1 / torch.sqrt((b * b).mean(1, keepdim=True) + EPS)
        bn, g = b * rb, 1.0 if gt is None else gt
        u = (RS * g * wp * torch.ones_like(x)).abs() * size
        close(got[1], db, rb * (u + bn.abs() * (u * bn.abs()).mean(1, keepdim=True)), args[0].dtype)
        close(got[3], dwp, (RS * (g * torch.ones_like(x)).abs() * size * bn.abs()).sum(0), torch.float32)
        if gt is not None:
            t = (RS * size * bn * wp).abs()
            close(got[2], dgate, t.sum(0) if gt.dim() == 1 else t.sum(1, keepdim=True), torch.float32)
    if dxn is not None:
        # y is itself a sum, of x and the branch: its error goes by their magnitudes
        close(got[4], dwn, (dxn.double().abs() * ry * (x.abs() + (y - x).abs())).sum(0), torch.float32)


SHAPES = [(1, 1), (1, 7), (3, 8), (2, 64), (5, 100), (9, 256), (33, 4096), (4, 4104), (3, 7168), (2, 8192), (2, 8200),
          (3, 16384), (2, 16383), (700, 64)]


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward_and_backward(T, H, dtype, gate):
    args, dy, dxn = inputs(T, H, dtype, gate, seed=T + H)
    check_forward(args, forward(args))
    check_backward(args, dy, dxn, backward(args, dy, dxn))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("block,pre,with_dy", [(False, True, True), (False, True, False), (True, False, True),
                                               (True, True, False)])
def test_parts(block, pre, with_dy, dtype):
    """Only the norm before, only the norm after, and no gradient of y."""
    for T, H in ((37, 384), (700, 40)):
        args, dy, dxn = inputs(T, H, dtype, "channel", block, pre, seed=5)
        check_forward(args, forward(args))
        dy = dy if with_dy else None
        check_backward(args, dy, dxn, backward(args, dy, dxn))


@pytest.mark.parametrize("dtype", list(DT))
def test_unaligned_streams_and_repeats(dtype):
    args, dy, dxn = inputs(50, 512, dtype, "channel", seed=6)
    side = torch.cuda.Stream()
    f, b = forward(args), backward(args, dy, dxn)
    assert all(torch.equal(u, v) for u, v in zip(f, forward(args, stream=side)))
    assert all(torch.equal(u, v) for u, v in zip(b, backward(args, dy, dxn, stream=side)))
    check_forward(args, forward(args, offset=1))
    check_backward(args, dy, dxn, backward(args, dy, dxn, offset=1))


def test_in_place():
    args, dy, dxn = inputs(20, 256, "bf16", "token", seed=7)
    want = forward(args)
    d = [dev(a) for a in args]
    xn = torch.empty_like(d[0])
    moe.moe_block_norm(*d, RS, EPS, d[0], xn)  # y over x
    assert torch.equal(d[0].cpu(), want[0]) and torch.equal(xn.cpu(), want[1])
    want = backward(args, dy, dxn)
    d, g, gn = [dev(a) for a in args], dev(dy), dev(dxn)
    db = torch.empty_like(g)
    ws = torch.empty(moe.moe_block_norm_workspace_bytes(20, 256), dtype=torch.uint8, device="cuda")
    moe.moe_block_norm_backward(*d, RS, EPS, g, gn, g, db, None, None, None, ws)  # dx over dy, no parameters' gradients
    assert torch.equal(g.cpu(), want[0]) and torch.equal(db.cpu(), want[1])


def test_zero_rows_and_extreme_values():
    """A zero row norms to zero; large rows keep finite statistics in fp32; NaN stays in its row."""
    args, dy, dxn = inputs(6, 128, "f32", "none", seed=8)
    args[0][1], args[1][1] = 0.0, 0.0
    args[0][2] *= 1e15
    args[1][3] *= 1e-20
    check_forward(args, forward(args))
    check_backward(args, dy, dxn, backward(args, dy, dxn))
    args[1][4, 5] = float("nan")
    y, xn = forward(args)
    assert torch.isnan(y[4]).all() and not torch.isnan(y[[0, 1, 2, 3, 5]]).any() and not torch.isnan(xn[5]).any()


def test_no_rows():
    args, dy, dxn = inputs(0, 64, "f32", "channel")
    y, xn = forward(args)
    assert y.shape == (0, 64)
    dx, db, dgate, dwp, dwn = backward(args, dy, dxn)
    assert all((t == 0).all() for t in (dgate, dwp, dwn))


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_gradient_against_differences(gate):
    """Central differences of <dy, y> + <dxn, xn> in 64 bits along random directions of every input."""
    args, dy, dxn = inputs(7, 48, "f32", gate, seed=11)
    grads = backward(args, dy, dxn)
    a = [None if t is None else t.double() for t in args]
    gen = torch.Generator().manual_seed(1)

    def value(v):
        y, xn = ref.block_norm(*v, RS, EPS)
        return float((y * dy.double()).sum() + (xn * dxn.double()).sum())

    for i, g in enumerate(grads):
        if g is None:
            continue
        d = torch.randn(a[i].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        slope = (value(a[:i] + [a[i] + h * d] + a[i + 1:]) - value(a[:i] + [a[i] - h * d] + a[i + 1:])) / (2 * h)
        assert abs(float((g.double() * d).sum()) - slope) <= 1e-4 * float((g.double() * d).abs().sum()) + 1e-6


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,H", [(1000, 4096), (640, 7168), (500, 8200), (900, 384), (3000, 40), (460, 12288)])
def test_more_rows_than_ctas(T, H, dtype):
    """Rows fetched ahead: several rows a CTA, at each number of rows in flight."""
    for gate, block in (("channel", True), ("token", True), ("none", False)):
        args, dy, dxn = inputs(T, H, dtype, gate, block, seed=T)
        check_forward(args, forward(args))
        check_backward(args, dy, dxn, backward(args, dy, dxn))


def test_two_host_threads_of_different_row_lengths():
    """Rows of two lengths that one kernel serves with different amounts of shared memory, called from two threads."""
    import threading
    T, calls = 160, 4000  # more rows than SMs: they are fetched ahead into shared memory
    jobs = []
    for H in (8192, 4352):
        g = torch.Generator(device="cuda").manual_seed(H)
        x = torch.randn(T, H, generator=g, device="cuda")
        w = torch.randn(H, generator=g, device="cuda")
        y, xn = torch.empty_like(x), torch.empty_like(x)
        moe.moe_block_norm(x, x, None, w, w, 1.0, 1e-6, y, xn)
        jobs.append((x, w, y, xn, y.clone(), xn.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed = []

    def work(x, w, y, xn, want_y, want_xn, stream):
        try:
            for _ in range(calls):
                moe.moe_block_norm(x, x, None, w, w, 1.0, 1e-6, y, xn, stream)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for x, w, y, xn, want_y, want_xn, _ in jobs:
        assert torch.equal(y, want_y) and torch.equal(xn, want_xn)
