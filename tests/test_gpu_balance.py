"""The router's balance loss and its gradient against 64 bits and against differences of the loss.

Bounds.  Counts are equal.  A score's relative error is at most 2^-18 (the exponential of an argument up to 30 in
magnitude rounded to 24 bits, its own 2^-22, the sum and the division), sums of scores keep it, and so does the loss (a sum
of positive terms).  The gradient p (v - mean v) has that error in p and, in the difference, 2^-18 of the largest
|v - mean|; both are at most 2^-16 of p max|v - mean|."""
import pytest
import torch

import operator_reference as ref
import routed_expert_layer_moe_gb300 as moe

pytestmark = pytest.mark.gpu

REL = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def built():
    from routed_expert_layer_moe_gb300 import build
    build.build()
    torch.cuda.init()


def run(logits, ids, valid, seq, score, coef, dloss, stream=None, offset=0):
    T, E = logits.shape
    K = ids.shape[1]
    B = 1 if seq is None else len(seq) - 1
    p = moe.Problem.make(T=T, H=128, I=128, E=E, K=K, layout="contig")
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731

    def shifted(t):  # the same values at an address that is only 4-byte aligned
        if not offset:
            return t.cuda()
        buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
        buf[offset:] = t.reshape(-1).cuda()
        return buf[offset:].view(t.shape)

    lg = shifted(logits)
    seqd = None if seq is None else torch.tensor(seq, dtype=torch.int32, device="cuda")
    out = dict(loss=torch.full((B,), -7.0, device="cuda"),
               counts=torch.full((B, E), -7, dtype=torch.int32, device="cuda"),
               prob_sum=torch.full((B, E), -7.0, device="cuda"),
               tokens=torch.full((B,), -7, dtype=torch.int32, device="cuda"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((moe.moe_balance_workspace_bytes(p, B),), 0xA5, dtype=torch.uint8, device="cuda")
    dlogits = shifted(torch.full((T, E), -7.0))
    ids, valid, dl = cu(ids), cu(valid), cu(dloss)
    torch.cuda.synchronize()
    moe.moe_balance_loss(p, lg, ids, valid, seqd, score, coef, *out.values(), err, ws, stream=stream)
    moe.moe_balance_loss_backward(p, lg, valid, seqd, score, coef, out["counts"], out["tokens"], dl, dlogits,
                                  stream=stream)
    torch.cuda.synchronize()
    return {**{k: v.cpu() for k, v in out.items()}, "dlogits": dlogits.cpu(), "err": int(err)}


def check(got, want, logits, ids, valid, seq, score, coef, dloss):
    T, E = logits.shape
    K = ids.shape[1]
    assert torch.equal(got["counts"].long(), want["counts"]) and torch.equal(got["tokens"].long(), want["tokens"])
    for k in ("prob_sum", "loss"):
        assert ((got[k].double() - want[k]).abs() <= REL * want[k].abs() + 1e-37).all(), k
    seqs = [0, T] if seq is None else seq
    bound = torch.zeros(T, E, dtype=torch.float64)
    for b in range(len(seqs) - 1):
        rows = slice(seqs[b], seqs[b + 1])
        n = max(int(want["tokens"][b]), 1)
        v = want["counts"][b].double()
        v = (v - v.mean()).abs().max() * coef * E / (K * n * n) * abs(float(dloss[b]))
        a = logits[rows].double()
        p = torch.softmax(a, 1) if score == "softmax" else torch.sigmoid(a) / torch.sigmoid(a).sum(1, keepdim=True)
        bound[rows] = 2.0 ** -16 * torch.nan_to_num(p) * v
    d = (got["dlogits"].double() - want["dlogits"]).abs()
    assert (d <= bound + 1e-37).all(), (d - bound).max()


def inputs(T, E, K, seed=0, off=0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) * 1.5 + torch.randn(E, generator=g)
    if off:
        logits[:, torch.randperm(E, generator=g)[:off]] = -float("inf")
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int() if T else \
        torch.zeros(0, K, dtype=torch.int32)
    return logits, ids, g


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K,seq", [
    (1, 8, 2, None), (1, 1, 1, None), (5, 3, 3, None), (40, 33, 4, None), (300, 256, 8, None), (64, 512, 10, None),
    (70, 513, 6, None), (33, 1024, 32, None), (20, 1023, 1, None), (129, 128, 4, None), (50, 129, 2, None),
    (100, 64, 4, [0, 1, 1, 40, 99, 100]),            # an empty segment, segments of one token
    (100, 20, 3, [0, 0, 0, 100, 100]),               # empty first and last ones
    (90, 260, 5, [7, 30, 31, 80]),                   # tokens outside every segment
    (2600, 16, 2, [0, 3, 1000, 1001, 2590, 2600]),   # tiles that several segments meet
])
def test_against_64_bits(T, E, K, seq, score):
    logits, ids, g = inputs(T, E, K, seed=T + E, off=E // 8)
    B = 1 if seq is None else len(seq) - 1
    dloss = torch.randn(B, generator=g)
    for valid in (None, (torch.rand(T, generator=g) < 0.7).to(torch.uint8)):
        args = (logits, ids, valid, seq, score, 0.01, dloss)
        got = run(*args)
        assert got["err"] == 0
        check(got, ref.balance(*args), *args)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score):
    """(loss(l + h d) - loss(l - h d)) / 2h along random directions, in 64 bits, with the counts held."""
    T, E, K, coef = 24, 12, 3, 0.5
    logits, ids, g = inputs(T, E, K, seed=9)
    dloss = torch.tensor([1.3, -0.4])
    seq = [0, 10, 24]
    got = run(logits, ids, None, seq, score, coef, dloss)["dlogits"].double()

    def loss(l):
        r = ref.balance(l, ids, None, seq, score, coef, dloss)
        return float((r["loss"] * dloss.double()).sum())

    for _ in range(5):
        d = torch.randn(T, E, generator=g, dtype=torch.float64)
        h = 1e-4  # the third-order term: below 1e-8 of the slope
        slope = (loss(logits.double() + h * d) - loss(logits.double() - h * d)) / (2 * h)
        assert abs(float((got * d).sum()) - slope) <= 1e-4 * float((got * d).abs().sum())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_tokens_and_switched_off_experts(score):
    """A masked token's logits and ids are not read; a row with every expert off counts but has no scores."""
    T, E, K = 37, 40, 4
    logits, ids, g = inputs(T, E, K, seed=4)
    valid = torch.ones(T, dtype=torch.uint8)
    valid[[0, 9, 36]] = 0
    logits[0], logits[9, 3] = float("nan"), float("inf")
    ids[36] = 1 << 30
    logits[5] = -float("inf")
    logits[6, 1:] = -float("inf")
    clean = logits.clone()
    clean[valid == 0] = 0.0
    dloss = torch.tensor([1.0])
    got = run(logits, ids, valid, None, score, 0.1, dloss)
    args = (clean, ids, valid, None, score, 0.1, dloss)
    assert got["err"] == 0
    check(got, ref.balance(*args), *args)
    assert (got["dlogits"][[0, 9, 36, 5]] == 0).all()


def test_all_tokens_masked_and_no_tokens():
    for T in (0, 50):
        logits, ids, _ = inputs(T, 8, 2)
        got = run(logits, ids, torch.zeros(T, dtype=torch.uint8), [0, T // 2, T], "softmax", 1.0, torch.ones(2))
        assert got["err"] == 0
        for k in ("loss", "counts", "prob_sum", "tokens", "dlogits"):
            assert (got[k] == 0).all(), k


def test_bad_ids_are_flagged_and_not_counted():
    logits, ids, _ = inputs(20, 8, 2)
    ids[3, 0], ids[7, 1] = 8, -1
    got = run(logits, ids, None, None, "softmax", 1.0, torch.ones(1))
    assert got["err"] == moe.MOE_FLAG_BAD_EXPERT
    args = (logits, ids, None, None, "softmax", 1.0, torch.ones(1))
    check(got, ref.balance(*args), *args)


def test_nan_logits_show():
    logits, ids, _ = inputs(20, 8, 2)
    logits[4, 4] = float("nan")
    got = run(logits, ids, None, [0, 10, 20], "softmax", 1.0, torch.ones(2))
    assert torch.isnan(got["loss"][0]) and not torch.isnan(got["loss"][1])
    assert torch.isnan(got["dlogits"][4]).all() and not torch.isnan(got["dlogits"][:4]).any()


def test_unaligned_rows_other_streams_and_repeats():
    logits, ids, g = inputs(777, 64, 4, seed=2)
    args = (logits, ids, None, [0, 100, 777], "softmax", 0.01, torch.tensor([1.0, 2.0]))
    a = run(*args)
    side = torch.cuda.Stream()
    for other in (run(*args), run(*args, stream=side)):
        for k in a:
            assert a[k] == other[k] if k == "err" else torch.equal(a[k], other[k]), k
    b = run(*args, offset=1)  # 4-byte aligned rows
    check(b, ref.balance(*args), *args)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,seq", [
    (10, [5, 5, 10]), (10, [3, 3, 3, 10]), (80, [7, 7, 30, 80]),  # one launch
    (100, [40, 40, 40, 100]), (200, [100, 100, 170]),             # the first segment with tokens in a later tile
    (50, [20, 20]), (50, [50, 50, 50]),                           # no segment has tokens
    (900, [7, 7, 30, 880]), (900, [400, 400, 400, 900]),          # two kernels
    (900, [33] * 80 + [500, 500, 501, 890]),                      # more empty segments than a look-up holds
])
def test_empty_segments_behind_tokens_of_no_segment(T, seq, score):
    """Tokens before the first segment, and that one empty: the segments after it keep their tokens."""
    logits, ids, g = inputs(T, 24, 3, seed=T)
    dloss = torch.randn(len(seq) - 1, generator=g)
    for valid in (None, (torch.rand(T, generator=g) < 0.7).to(torch.uint8)):
        args = (logits, ids, valid, seq, score, 0.01, dloss)
        got = run(*args)
        assert got["err"] == 0
        check(got, ref.balance(*args), *args)


@pytest.mark.parametrize("E", [6, 64, 257, 512, 1000])
def test_softmax_rows_of_large_logits(E):
    """Logits of any finite size, the type's lowest value in a whole row among them: a row of equal ones is uniform."""
    big = torch.finfo(torch.float32).max
    tops = [big, 1e30, 1e10, 2.0 ** 25, 1e5, -1e5, -(2.0 ** 25), -1e10, -1e30, -big]
    T, K = 3 * len(tops), min(E, 4)
    g = torch.Generator().manual_seed(E)
    logits = torch.empty(T, E)
    for i, top in enumerate(tops):
        logits[3 * i] = top
        logits[3 * i + 1] = max(top, -big) - torch.rand(E, generator=g) * 20.0
        logits[3 * i + 2] = -big                   # masked with the lowest value, a few experts left
        logits[3 * i + 2, :3] = top
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int()
    args = (logits, ids, None, [0, 17, T], "softmax", 0.01, torch.tensor([1.0, -2.0]))
    got = run(*args)
    assert got["err"] == 0
    check(got, ref.balance(*args), *args)


@pytest.mark.parametrize("E", [5, 48, 256, 300, 700])
def test_sigmoid_rows_of_low_logits(E):
    """Rows whose largest logit is far below zero, where sigmoid(l) itself is below the smallest normal number: the scores
    still sum to one.  Bound: 2^-16.  Where the sigmoid is taken directly its exponential's argument is at most 126,
    rounded to 2^-18 and with log2 e's own rounding 2^-20 off; times ln 2, with the exponential, the reciprocal, the
    sum and the division, under 2^-17.  Ratios of exponentials of differences up to 30 are better than that."""
    tops = [-20.0, -52.0, -55.0, -55.4, -56.0, -60.0, -80.0, -87.0, -88.0, -100.0, -104.0, -150.0, -1e4, -1e30]
    T, K = len(tops) * 3, min(E, 4)
    g = torch.Generator().manual_seed(E)
    logits = torch.empty(T, E)
    for i, top in enumerate(tops):
        spread = torch.rand(E, generator=g) * 30.0
        logits[3 * i] = top                       # all alike
        logits[3 * i + 1] = top - spread          # the largest and others below it
        logits[3 * i + 1, i % E] = top
        logits[3 * i + 2] = top - spread
        logits[3 * i + 2, ::2] = -float("inf")    # and experts that are off
        logits[3 * i + 2, -1 if E % 2 == 0 else 1] = top
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int()
    perm = torch.randperm(T, generator=g)         # neighbours of every kind in a warp
    logits, ids = logits[perm], ids[perm]
    dloss = torch.tensor([1.0, -2.0])
    seq = [0, T // 2, T]
    # the reference's sigmoid in 64 bits underflows below -745: there its ratios are those of the differences
    exact_logits, top = logits.double(), logits.double().amax(1, keepdim=True)
    exact_logits = torch.where(top < -700, exact_logits - top - 100.0, exact_logits)
    for valid in (None, (torch.rand(T, generator=g) < 0.7).to(torch.uint8)):
        got = run(logits, ids, valid, seq, "sigmoid", 0.01, dloss)
        want = ref.balance(exact_logits, ids, valid, seq, "sigmoid", 0.01, dloss)
        assert got["err"] == 0 and torch.equal(got["counts"].long(), want["counts"])
        for k in ("prob_sum", "loss"):
            assert ((got[k].double() - want[k]).abs() <= 2.0 ** -16 * want[k].abs() + 1e-37).all(), k
        p = torch.sigmoid(exact_logits)
        p = p / p.sum(1, keepdim=True)
        for b in range(2):
            rows, n = slice(seq[b], seq[b + 1]), max(int(want["tokens"][b]), 1)
            v = want["counts"][b].double()
            v = (v - v.mean()).abs().max() * 0.01 * E / (K * n * n) * abs(float(dloss[b]))
            # p and the difference v - sum v p each carry the scores' error, the difference of both signs
            d = (got["dlogits"][rows].double() - want["dlogits"][rows]).abs()
            assert (d <= 2.0 ** -14 * p[rows] * v + 1e-37).all()
