"""Arguments that the training calls and the 8-bit checkpoints refuse, on the host, before any launch."""
import ctypes

import pytest
import torch

import routed_expert_layer_moe_gb300 as moe
from routed_expert_layer_moe_gb300 import build as moe_build

INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID, moe.MOE_ERR_UNSUPPORTED
A = 4096  # an aligned address that is never followed: every call here is refused on the host
F32, BF16 = moe.MOE_F32, moe.MOE_BF16


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe_build.build()
    return moe.lib()


def problem(**kw):
    return moe.Problem.make(**{**dict(T=4, H=256, I=128, E=8, K=2, layout="contig"), **kw})


def test_fp8(lib):
    for f in (lib.moe_fp8_quantize, lib.moe_fp8_dequantize):
        assert f(F32, 0, 32, None, None, None, None) == moe.MOE_OK  # nothing to do
        assert f(BF16, 4, 0, None, None, None, None) == moe.MOE_OK
        for bad in (moe.MOE_E4M3, 7, -1):
            assert f(bad, 4, 32, A, A, A, None) == INVALID
        assert f(F32, -1, 32, A, A, A, None) == f(F32, 4, -1, A, A, A, None) == INVALID
        assert f(F32, 1 << 34, 1, A, A, A, None) == f(F32, 1, 1 << 34, A, A, A, None) == INVALID
        assert f(F32, 1 << 30, 1 << 20, A, A, A, None) == INVALID
        for null in range(3):
            assert f(BF16, 4, 33, *[None if i == null else A for i in range(3)], None) == INVALID


    # x, codes, scales and codes, scales, out: values and scales at their own size's alignment, codes anywhere
    assert lib.moe_fp8_quantize(F32, 4, 33, A + 2, A, A, None) == UNSUPPORTED
    assert lib.moe_fp8_quantize(BF16, 4, 33, A + 1, A, A, None) == UNSUPPORTED
    assert lib.moe_fp8_quantize(BF16, 4, 33, A, A, A + 2, None) == UNSUPPORTED
    assert lib.moe_fp8_dequantize(F32, 4, 33, A, A, A + 2, None) == UNSUPPORTED
    assert lib.moe_fp8_dequantize(BF16, 4, 33, A, A, A + 1, None) == UNSUPPORTED
    assert lib.moe_fp8_dequantize(BF16, 4, 33, A, A + 2, A, None) == UNSUPPORTED


@pytest.mark.parametrize("wt,act,out", [("f32", "f32", "f32"), ("e4m3", "bf16", "bf16"), ("e2m1", "bf16", "bf16"),
                                        ("mxfp4", "bf16", "bf16")])
def test_other_experts(lib, wt, act, out):
    p = problem(wt=wt, act=act, out=out)
    assert moe.moe_check_problem(p) == moe.MOE_OK
    q = ctypes.byref(p)
    assert lib.moe_grouped_swiglu_gemm_save(q, *[A] * 8, None) == UNSUPPORTED
    assert lib.moe_combine_backward(q, *[A] * 7, None) == UNSUPPORTED
    assert lib.moe_grouped_ffn_backward(q, *[A] * 14, BF16, 0, A, None) == UNSUPPORTED
    assert lib.moe_permute_backward(q, *[A] * 3, None) == UNSUPPORTED
    assert lib.moe_layer_backward(q, *[A] * 12, 0, A, 1, 1.0, *[A] * 11, BF16, 0, A, None) == UNSUPPORTED
    for call in (lambda: moe.moe_grouped_swiglu_gemm_save(p, *[None] * 8), lambda: moe.moe_permute_backward(p, *[None] * 3),
                 lambda: moe.MoeLayer(p, act, wt, out, None, None, device="cpu", train=True)):
        with pytest.raises(moe.MoeError):
            call()


def test_bad_problems(lib):
    p = problem(K=9)
    q = ctypes.byref(p)
    assert lib.moe_grouped_swiglu_gemm_save(q, *[A] * 8, None) == INVALID
    assert lib.moe_layer_backward(q, *[A] * 12, 0, A, 1, 1.0, *[A] * 11, BF16, 0, A, None) == INVALID
    assert lib.moe_route_backward(q, 0, *[A] * 4, 1, 1.0, A, A, None) == INVALID
    # rows of weights past 32 bits
    p = problem(E=1024, I=1 << 21, H=128)
    assert moe.moe_check_problem(p) == moe.MOE_OK
    assert lib.moe_grouped_swiglu_gemm_save(ctypes.byref(p), *[A] * 8, None) == UNSUPPORTED


def each_null(call, n, skip=()):
    return {i: call(*[None if i == k else A for k in range(n)]) for i in range(n) if i not in skip}


def test_null_and_unaligned(lib):
    q = ctypes.byref(problem())
    up = lambda *a: lib.moe_grouped_swiglu_gemm_save(q, *a, None)  # noqa: E731
    assert set(each_null(up, 8).values()) == {INVALID}
    for i, off in ((0, 8), (1, 8), (4, 8), (5, 8), (6, 2)):  # xg, w13, hg, gu, gu_scales
        assert up(*[A + off if i == k else A for k in range(8)]) == UNSUPPORTED, i
    cb = lambda *a: lib.moe_combine_backward(q, *a, None)  # noqa: E731
    assert set(each_null(cb, 7, skip=(6,)).values()) == {INVALID}
    for i in (0, 1, 4):
        assert cb(*[A + 8 if i == k else A for k in range(7)]) == UNSUPPORTED, i
    ffn = lambda *a, dt=BF16, acc=0: lib.moe_grouped_ffn_backward(q, *a, dt, acc, A, None)  # noqa: E731
    # dyg, wg, xg, w13, w2, gu, gu_scales, masked_m, offsets, dgu, hg, dxg, dw13, dw2
    optional = (1, 11, 12, 13)
    assert set(each_null(ffn, 14, skip=optional).values()) == {INVALID}
    for i in (0, 2, 3, 4, 5, 9, 10, 11, 12, 13):
        assert ffn(*[A + 8 if i == k else A for k in range(14)]) == UNSUPPORTED, i
    for i in (1, 6):
        assert ffn(*[A + 2 if i == k else A for k in range(14)]) == UNSUPPORTED, i
    assert ffn(*[A] * 14, dt=moe.MOE_E4M3) == INVALID
    assert ffn(*[A] * 14, acc=1) == UNSUPPORTED  # sums go on in fp32 alone
    assert lib.moe_grouped_ffn_backward(q, *[A] * 14, BF16, 0, None, None) == INVALID
    pb = lambda *a: lib.moe_permute_backward(q, *a, None)  # noqa: E731
    assert set(each_null(pb, 3).values()) == {INVALID}
    assert pb(A + 8, A, A) == pb(A, A, A + 8) == UNSUPPORTED
    rb = lambda *a, score=0: lib.moe_route_backward(q, score, *a[:4], 1, 1.0, *a[4:], None)  # noqa: E731
    # logits, ids, w, dw, add, dlogits
    assert {i for i, r in each_null(rb, 6, skip=(0, 4)).items() if r == INVALID} == {1, 2, 3, 5}
    assert rb(None, A, A, A, None, A, score=1) == INVALID  # sigmoid scores need the logits
    assert rb(*[A] * 6, score=2) == rb(*[A] * 6, score=-1) == INVALID
    # dout, yg, row_of, ids, w, xg, w13, w2, gu, gu_scales, masked_m, offsets | score, logits, renormalize, scale |
    # add, dyg, wg, dgu, hg, dxg, dw, dx, dlogits, dw13, dw2
    lb = lambda *a, score=0, logits=A: lib.moe_layer_backward(q, *a[:12], score, logits, 1, 1.0, *a[12:], BF16, 0, A, None)  # noqa: E731
    assert set(each_null(lb, 23, skip=(12, 21, 22)).values()) == {INVALID}
    assert lb(*[A] * 23, score=1, logits=None) == INVALID and lb(*[A] * 23, score=3) == INVALID
    for i in (0, 1, 5, 6, 7, 8, 13, 15, 16, 17, 19, 21, 22):
        assert lb(*[A + 8 if i == k else A for k in range(23)]) == UNSUPPORTED, i


def test_nothing_to_do(lib):
    q = ctypes.byref(problem(T=0))
    assert lib.moe_grouped_swiglu_gemm_save(q, *[None] * 9) == moe.MOE_OK
    assert lib.moe_combine_backward(q, *[None] * 8) == moe.MOE_OK
    assert lib.moe_permute_backward(q, *[None] * 4) == moe.MOE_OK
    assert lib.moe_route_backward(q, 0, *[None] * 4, 1, 1.0, *[None] * 3) == moe.MOE_OK
    assert lib.moe_grouped_ffn_backward(q, *[None] * 14, BF16, 0, None, None) == moe.MOE_OK


def test_tensors(lib):
    p = problem()
    cpu = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_fp8_quantize(cpu, torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        moe.moe_fp8_quantize(cpu.half(), None, None)
    with pytest.raises(ValueError, match="dxg"):
        moe.moe_permute_backward(p, torch.zeros(8, 256), torch.zeros(4, 2, dtype=torch.int32), cpu)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        moe.moe_grouped_ffn_backward(p, *[None] * 12, torch.zeros(1, dtype=torch.float16), None, None)
    with pytest.raises(KeyError):
        moe.moe_route_backward(p, "argmax", None, None, None, None, None)
