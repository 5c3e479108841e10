"""Arguments that the MXFP4, balance-loss and block-norm calls refuse, on the host, before any launch."""
import ctypes

import pytest
import torch

import routed_expert_layer_moe_gb300 as moe
from routed_expert_layer_moe_gb300 import build as moe_build

INVALID, UNSUPPORTED, WORKSPACE = moe.MOE_ERR_INVALID, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
A = 4096         # an aligned address that is never followed: every call here is refused on the host
F32, BF16 = moe.MOE_F32, moe.MOE_BF16


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe_build.build()
    return moe.lib()


def test_mx_conversions(lib):
    for f in (lib.moe_mx_quantize, lib.moe_mx_dequantize):
        assert f(F32, 0, 32, None, None, None, None) == moe.MOE_OK  # nothing to do
        assert f(F32, 4, 0, None, None, None, None) == moe.MOE_OK
        assert f(moe.MOE_E4M3, 4, 32, A, A, A, None) == INVALID
        assert f(F32, -1, 32, A, A, A, None) == INVALID
        assert f(F32, 4, 48, A, A, A, None) == INVALID
        assert f(F32, 4, -32, A, A, A, None) == INVALID
        assert f(F32, 1 << 40, 1 << 30, A, A, A, None) == INVALID
        for null in range(3):
            assert f(BF16, 4, 32, *[None if i == null else A for i in range(3)], None) == INVALID
    assert lib.moe_mx_quantize(F32, 4, 32, A + 8, A, A, None) == UNSUPPORTED   # values: 16 bytes
    assert lib.moe_mx_quantize(F32, 4, 32, A, A + 2, A, None) == UNSUPPORTED   # codes: 4 bytes
    assert lib.moe_mx_dequantize(BF16, 4, 32, A + 2, A, A, None) == UNSUPPORTED
    assert lib.moe_mx_dequantize(BF16, 4, 32, A, A, A + 2, None) == UNSUPPORTED


def test_mxfp4_problems(lib):
    def p(**kw):
        return moe.Problem.make(**{**dict(T=4, H=256, I=256, E=8, K=2, M_max=4, wt="mxfp4"), **kw})

    assert moe.moe_check_problem(p()) == moe.MOE_OK
    assert moe.moe_gemm_tile_rows(p(), 3) == moe.moe_gemm_tile_rows(p(), 4) == 128
    assert moe.moe_check_problem(p(H=192)) == UNSUPPORTED
    assert moe.moe_check_problem(p(I=64)) == UNSUPPORTED
    assert moe.moe_check_problem(p(act="f32", out="f32")) == UNSUPPORTED
    assert moe.moe_check_problem(p(out="f32")) == UNSUPPORTED
    q = p()
    q.wt = 5
    assert moe.moe_check_problem(q) == INVALID
    q = ctypes.byref(p())
    ws = moe.moe_workspace_bytes(p())
    gate = lambda *a: lib.moe_grouped_swiglu_gemm(q, *a, A, ws, None)  # noqa: E731
    # xg, xg_scales, w13, w13_scales, masked_m, offsets, hg, hg_scales, err_flag
    good = [A] * 9
    for i in range(9):
        assert gate(*good[:i], None, *good[i + 1:]) == INVALID, i
    for i, off in ((0, 8), (2, 8), (6, 8), (1, 2), (3, 1), (7, 2)):
        assert gate(*good[:i], A + off, *good[i + 1:]) == UNSUPPORTED, i
    assert lib.moe_grouped_swiglu_gemm(q, *good, A, ws - 1, None) == WORKSPACE
    assert lib.moe_grouped_down_gemm(q, A, A + 1, A, A, A, A, A, A, A, ws, None) == UNSUPPORTED
    assert lib.moe_grouped_ffn(q, A, A, A, A, A, A + 2, A, A, A, A, A, A, A, ws, None) == UNSUPPORTED
    assert lib.moe_ffn_combine(q, A, A, A, None, A, A, A, A, A, A, A, A, A, A, A, A, ws, None) == INVALID
    assert lib.moe_permute(q, A, A, None, A, A, A, A, A, None, A, A, ws, None) == INVALID  # no scales


def test_balance(lib):
    prob = moe.Problem.make(T=8, H=128, I=128, E=8, K=2, layout="contig")
    q, ws = ctypes.byref(prob), moe.moe_balance_workspace_bytes(prob, 2)
    assert ws > 0 and moe.moe_balance_workspace_bytes(prob, 0) == 0
    assert moe.moe_balance_workspace_bytes(prob, 65536) == 0

    def fwd(logits=A, ids=A, valid=None, seq=A, nseq=2, score=0, outs=(A, A, A, A), err=A, w=A, wb=ws, p=q):
        return lib.moe_balance_loss(p, logits, ids, valid, seq, nseq, score, 0.1, *outs, err, w, wb, None)

    assert fwd(p=None) == INVALID
    assert fwd(p=ctypes.byref(moe.Problem.make(T=8, H=128, I=128, E=2000, K=2, layout="contig"))) == INVALID
    for kw in (dict(logits=None), dict(ids=None), dict(seq=None), dict(nseq=0), dict(nseq=65536), dict(score=2),
               dict(score=-1), dict(err=None)):
        assert fwd(**kw) == INVALID, kw
    for i in range(4):
        assert fwd(outs=[None if j == i else A for j in range(4)]) == INVALID
    assert fwd(w=None) == WORKSPACE and fwd(wb=ws - 1) == WORKSPACE
    assert fwd(w=A + 4) == UNSUPPORTED

    def bwd(logits=A, seq=A, nseq=2, score=1, counts=A, tokens=A, dloss=A, out=A):
        return lib.moe_balance_loss_backward(q, logits, None, seq, nseq, score, 0.1, counts, tokens, dloss, out, None)

    for kw in (dict(logits=None), dict(seq=None), dict(nseq=0), dict(score=7), dict(counts=None), dict(tokens=None),
               dict(dloss=None), dict(out=None)):
        assert bwd(**kw) == INVALID, kw


def test_block_norm(lib):
    def fwd(dtype=BF16, T=4, H=64, x=A, block=A, kind=1, gate=A, w_post=A, w_pre=A, eps=1e-6, y=A, xn=A):
        return lib.moe_block_norm(dtype, T, H, x, block, kind, gate, w_post, w_pre, 1.0, eps, y, xn, None)

    assert fwd(T=0, x=None, block=None, y=None, xn=None) == moe.MOE_OK
    for kw in (dict(dtype=2), dict(T=-1), dict(H=0), dict(H=16385), dict(T=(1 << 30) + 1), dict(x=None), dict(kind=3), dict(kind=-1),
               dict(gate=None), dict(w_post=None), dict(w_pre=None), dict(xn=None), dict(y=None), dict(eps=-1.0),
               dict(eps=float("nan")), dict(block=None, y=None, xn=None, w_pre=None)):
        assert fwd(**kw) == INVALID, kw
    for k in ("x", "block", "gate", "w_post", "w_pre", "y", "xn"):
        assert fwd(**{k: A + 1}) == UNSUPPORTED, k
        assert fwd(dtype=F32, **{k: A + 2}) == UNSUPPORTED, k

    ws = moe.moe_block_norm_workspace_bytes(4, 64)
    assert ws > 0 and moe.moe_block_norm_workspace_bytes(4, 0) == 0 and moe.moe_block_norm_workspace_bytes(-1, 8) == 0

    def bwd(T=4, block=A, kind=1, gate=A, w_post=A, w_pre=A, dy=A, dxn=A, dx=A, dblock=A, dgate=A, dwp=A, dwn=A,
            w=A, wb=ws):
        return lib.moe_block_norm_backward(BF16, T, 64, A, block, kind, gate, w_post, w_pre, 1.0, 1e-6, dy, dxn, dx,
                                           dblock, dgate, dwp, dwn, w, wb, None)

    for kw in (dict(dx=None), dict(dblock=None), dict(block=None), dict(dxn=None), dict(w_pre=None),
               dict(w_pre=None, dxn=None, dy=None, dwn=None), dict(kind=0), dict(gate=None),
               dict(w_pre=None, dxn=None), dict(block=None, dblock=None, dgate=None)):
        assert bwd(**kw) == INVALID, kw
    for k in ("dy", "dxn", "dx", "dblock"):
        assert bwd(**{k: A + 1}) == UNSUPPORTED, k
    assert bwd(w=None) == WORKSPACE and bwd(wb=ws - 1) == WORKSPACE
    assert bwd(w=A + 2) == UNSUPPORTED


class Fake(torch.Tensor):
    """A CPU tensor that says it is on the GPU: the checks of the Python calls come before any launch."""

    @property
    def is_cuda(self):
        return True


def fake(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Fake)


def test_python_calls_check_types_shapes_and_layout():
    u8 = torch.uint8
    x, c, s = fake(4, 64), fake(4, 32, dtype=u8), fake(4, 2, dtype=u8)
    for bad in ((torch.zeros(4, 64), c, s), (fake(4, 64, dtype=torch.float16), c, s), (fake(4, 48), c, s),
                (x, fake(4, 33, dtype=u8), s), (x, fake(4, 32), s), (x, c, fake(4, 1, dtype=u8)),
                (fake(64, 4).t(), c, s), (fake(), c, s)):
        with pytest.raises(ValueError):
            moe.moe_mx_quantize(*bad)
        with pytest.raises(ValueError):
            moe.moe_mx_dequantize(bad[1], bad[2], bad[0])
    i32 = torch.int32
    p = moe.Problem.make(T=8, H=128, I=128, E=8, K=2, layout="contig")
    good = dict(logits=fake(8, 8), ids=fake(8, 2, dtype=i32), valid=None, seq_offsets=fake(3, dtype=i32),
                score="softmax", coef=1.0, loss=fake(2), counts=fake(2, 8, dtype=i32), prob_sum=fake(2, 8),
                tokens=fake(2, dtype=i32), err_flag=None, workspace=fake(4))
    for k, v in (("logits", fake(8, 9)), ("logits", fake(8, 16)[:, ::2]), ("logits", fake(8, 8, dtype=torch.bfloat16)),
                 ("ids", fake(8, 2, dtype=torch.int64)), ("valid", fake(8, dtype=torch.bool)),
                 ("seq_offsets", fake(1, dtype=i32)), ("loss", fake(1)), ("counts", fake(2, 8)),
                 ("tokens", fake(3, dtype=i32))):
        with pytest.raises(ValueError):
            moe.moe_balance_loss(p, **{**good, k: v})
    with pytest.raises(KeyError):
        moe.moe_balance_loss(p, **{**good, "score": "tanh"})
    ng = dict(x=x, block=x, gate=fake(64), w_post=fake(64), w_pre=fake(64), res_scale=1.0, eps=0.0, y=x, xn=x)
    for k, v in (("x", fake(4, 2, 32)), ("block", fake(4, 63)), ("gate", fake(4)), ("gate", fake(4, 2)),
                 ("w_post", fake(64, dtype=torch.bfloat16)), ("w_pre", fake(128)[::2]), ("y", fake(64, 4).t())):
        with pytest.raises(ValueError):
            moe.moe_block_norm(**{**ng, k: v})
