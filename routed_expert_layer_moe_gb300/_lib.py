"""ctypes binding of libmoe_gb300.so (the C ABI declared in include/moe.h).

Argument marshalling only: tensors become device pointers, the stream becomes
a cudaStream_t.  Every step runs in the library's CUDA kernels; there is no
other implementation to fall back to, so a missing library is an error."""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_gb300.so")

MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_WORKSPACE = 0, -1, -2, -3, -4
MOE_F32, MOE_BF16, MOE_E4M3, MOE_E2M1, MOE_MXFP4 = 0, 1, 2, 3, 4
MOE_LAYOUT_MASKED, MOE_LAYOUT_CONTIG = 0, 1
MOE_FLAG_OVERFLOW, MOE_FLAG_BAD_EXPERT, MOE_FLAG_BAD_MAP, MOE_FLAG_TIMEOUT = 1, 2, 4, 8
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN = 0, 1, 2
MOE_STATS_CTAS = 256                        # issue counters at the start of the workspace (include/moe.h)
MOE_STATS_BYTES = 2 * MOE_STATS_CTAS * 2 * 4

DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "e4m3": MOE_E4M3, "e2m1": MOE_E2M1, "mxfp4": MOE_MXFP4}
SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
LAYOUTS = {"masked": MOE_LAYOUT_MASKED, "contig": MOE_LAYOUT_CONTIG}

# every symbol include/moe.h declares
EXPORTS = ["moe_version", "moe_status_string", "moe_grouped_rows", "moe_workspace_bytes", "moe_check_problem",
           "moe_gemm_tile_rows",
           "moe_route_topk", "moe_route_grouped_topk", "moe_permute", "moe_permute_no_workspace",
           "moe_grouped_swiglu_gemm", "moe_grouped_down_gemm", "moe_grouped_ffn", "moe_combine",
           "moe_route_permute", "moe_ffn_combine",
           "moe_mx_quantize", "moe_mx_dequantize",
           "moe_balance_workspace_bytes", "moe_balance_loss", "moe_balance_loss_backward",
           "moe_block_norm_workspace_bytes", "moe_block_norm", "moe_block_norm_backward",
           "moe_eplb_record", "moe_eplb_rebalance", "moe_eplb_invert", "moe_selftest_bounded_wait"]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (where, status_string(status), status))


class Problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "H", "I", "E", "K", "P", "M_max", "has_shared", "act", "wt", "out", "layout")]

    @classmethod
    def make(cls, T, H, I, E, K, P=None, M_max=0, has_shared=0, act="bf16", wt="bf16", out="bf16",
             layout="masked") -> "Problem":
        return cls(T, H, I, E, K, E if P is None else P, M_max, has_shared, DTYPES[act], DTYPES[wt], DTYPES[out],
                   LAYOUTS[layout])

    def __repr__(self):
        return "Problem(%s)" % ", ".join("%s=%d" % (n, getattr(self, n)) for n, _ in self._fields_)


_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("%s is missing: build it with routed_expert_layer_moe_gb300.build.build() "
                          "(or __graft_entry__.build()); there is no other implementation" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    pp = ctypes.POINTER(Problem)
    L.moe_version.restype = i32
    L.moe_status_string.argtypes = [i32]
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_grouped_rows.argtypes = [pp]
    L.moe_grouped_rows.restype = i64
    L.moe_workspace_bytes.argtypes = [pp]
    L.moe_workspace_bytes.restype = sz
    L.moe_check_problem.argtypes = [pp]
    L.moe_check_problem.restype = i32
    L.moe_gemm_tile_rows.argtypes = [pp, i32]
    L.moe_gemm_tile_rows.restype = i32
    L.moe_route_topk.argtypes = [pp, vp, vp, vp, vp]
    L.moe_route_topk.restype = i32
    L.moe_route_grouped_topk.argtypes = [pp, vp, vp, i32, i32, i32, ctypes.c_float, vp, vp, vp]
    L.moe_route_grouped_topk.restype = i32
    L.moe_permute.argtypes = [pp] + [vp] * 11 + [sz, vp]
    L.moe_permute.restype = i32
    L.moe_permute_no_workspace.argtypes = [pp] + [vp] * 11
    L.moe_permute_no_workspace.restype = i32
    L.moe_grouped_swiglu_gemm.argtypes = [pp] + [vp] * 10 + [sz, vp]
    L.moe_grouped_swiglu_gemm.restype = i32
    L.moe_grouped_down_gemm.argtypes = [pp] + [vp] * 9 + [sz, vp]
    L.moe_grouped_down_gemm.restype = i32
    L.moe_grouped_ffn.argtypes = [pp] + [vp] * 13 + [sz, vp]
    L.moe_grouped_ffn.restype = i32
    L.moe_route_permute.argtypes = [pp] + [vp] * 13 + [sz, vp]
    L.moe_route_permute.restype = i32
    L.moe_ffn_combine.argtypes = [pp] + [vp] * 16 + [sz, vp]
    L.moe_ffn_combine.restype = i32
    L.moe_combine.argtypes = [pp, vp, vp, vp, vp, vp]
    L.moe_combine.restype = i32
    L.moe_eplb_record.argtypes = [pp, vp, i64, i32, vp, vp]
    L.moe_eplb_record.restype = i32
    L.moe_eplb_rebalance.argtypes = [pp, vp, i32, vp, vp, vp, vp, vp]
    L.moe_eplb_rebalance.restype = i32
    f32 = ctypes.c_float
    L.moe_mx_quantize.argtypes = [i32, i64, i64, vp, vp, vp, vp]
    L.moe_mx_quantize.restype = i32
    L.moe_mx_dequantize.argtypes = [i32, i64, i64, vp, vp, vp, vp]
    L.moe_mx_dequantize.restype = i32
    L.moe_balance_workspace_bytes.argtypes = [pp, i32]
    L.moe_balance_workspace_bytes.restype = sz
    L.moe_balance_loss.argtypes = [pp] + [vp] * 4 + [i32, i32, f32] + [vp] * 6 + [sz, vp]
    L.moe_balance_loss.restype = i32
    L.moe_balance_loss_backward.argtypes = [pp] + [vp] * 3 + [i32, i32, f32] + [vp] * 5
    L.moe_balance_loss_backward.restype = i32
    L.moe_block_norm_workspace_bytes.argtypes = [i32, i32]
    L.moe_block_norm_workspace_bytes.restype = sz
    L.moe_block_norm.argtypes = [i32, i32, i32, vp, vp, i32, vp, vp, vp, f32, f32, vp, vp, vp]
    L.moe_block_norm.restype = i32
    L.moe_block_norm_backward.argtypes = [i32, i32, i32, vp, vp, i32, vp, vp, vp, f32, f32] + [vp] * 8 + [sz, vp]
    L.moe_block_norm_backward.restype = i32
    L.moe_selftest_bounded_wait.argtypes = [i64, vp, vp]
    L.moe_selftest_bounded_wait.restype = i32
    L.moe_eplb_invert.argtypes = [i32, i32, vp, i32, vp, vp]
    L.moe_eplb_invert.restype = i32
    _lib = L
    return L


def status_string(s: int) -> str:
    return lib().moe_status_string(s).decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


# The current stream's handle without a stream object (2.8 us of a call's 10 us on a Grace core), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _allocate_on(stream):
    """Context in which torch allocates on the stream of a call: memory of a result that is dropped then goes back to
    that stream, behind the kernel that writes it.  stream: as the calls take it (None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        # 0 and 1 are the default stream's handles
        stream = torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


_FLOAT_DTYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def _arg(t, name: str, dtype, shape):
    """Device address of a dense tensor of this type and shape (None: no tensor); a ValueError otherwise.
    The calls below take whole arrays and no strides, so a view that is not dense would be read wrongly."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError("%s: expected a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s: expected a dense row-major tensor" % name)
    raise ValueError("%s: expected %s %s, got %s %s" % (name, dtype, tuple(shape), t.dtype, tuple(t.shape)))


def _values(t, name: str):
    """(moe_dtype, device address) of a dense float32 or bfloat16 tensor."""
    d = _FLOAT_DTYPES.get(t.dtype)
    if d is None:
        raise ValueError("%s: expected float32 or bfloat16, got %s" % (name, t.dtype))
    if t.is_cuda and t.is_contiguous():
        return d, t.data_ptr()
    return d, _arg(t, name, t.dtype, t.shape)


def moe_version() -> int:
    return lib().moe_version()


def moe_check_problem(p: Problem) -> int:
    return lib().moe_check_problem(ctypes.byref(p))


def moe_gemm_tile_rows(p: Problem, step: int) -> int:
    return lib().moe_gemm_tile_rows(ctypes.byref(p), step)


def moe_grouped_rows(p: Problem) -> int:
    return lib().moe_grouped_rows(ctypes.byref(p))


def moe_workspace_bytes(p: Problem) -> int:
    return lib().moe_workspace_bytes(ctypes.byref(p))


def moe_route_topk(p: Problem, logits, ids, w, stream=None) -> None:
    _check(lib().moe_route_topk(ctypes.byref(p), _ptr(logits), _ptr(ids), _ptr(w), _stream(stream)),
           "moe_route_topk")


def moe_route_grouped_topk(p: Problem, logits, bias, n_group: int, topk_group: int, ids, w, renormalize=True,
                           scale: float = 1.0, stream=None) -> None:
    _check(lib().moe_route_grouped_topk(ctypes.byref(p), _ptr(logits), _ptr(bias), n_group, topk_group,
                                        int(bool(renormalize)), float(scale), _ptr(ids), _ptr(w), _stream(stream)),
           "moe_route_grouped_topk")


def moe_permute(p: Problem, ids, x, phys_to_log, masked_m, offsets, row_of, src_of, xg, xg_scales, err_flag,
                workspace, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().moe_permute(ctypes.byref(p), _ptr(ids), _ptr(x), _ptr(phys_to_log), _ptr(masked_m),
                             _ptr(offsets), _ptr(row_of), _ptr(src_of), _ptr(xg), _ptr(xg_scales),
                             _ptr(err_flag), _ptr(workspace), nbytes, _stream(stream)), "moe_permute")


def moe_permute_no_workspace(p: Problem, ids, x, phys_to_log, masked_m, offsets, row_of, src_of, xg, xg_scales,
                             err_flag, stream=None) -> None:
    """moe_permute without a workspace argument, for callers that cannot allocate
    device memory; its scratch is a fixed array inside the library (see moe.h)."""
    _check(lib().moe_permute_no_workspace(ctypes.byref(p), _ptr(ids), _ptr(x), _ptr(phys_to_log), _ptr(masked_m),
                                          _ptr(offsets), _ptr(row_of), _ptr(src_of), _ptr(xg), _ptr(xg_scales),
                                          _ptr(err_flag), _stream(stream)), "moe_permute_no_workspace")


def moe_grouped_swiglu_gemm(p: Problem, xg, xg_scales, w13, w13_scales, masked_m, offsets, hg, hg_scales,
                            err_flag, workspace, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().moe_grouped_swiglu_gemm(ctypes.byref(p), _ptr(xg), _ptr(xg_scales), _ptr(w13), _ptr(w13_scales),
                                         _ptr(masked_m), _ptr(offsets), _ptr(hg), _ptr(hg_scales), _ptr(err_flag),
                                         _ptr(workspace), nbytes, _stream(stream)), "moe_grouped_swiglu_gemm")


def moe_grouped_down_gemm(p: Problem, hg, hg_scales, w2, w2_scales, masked_m, offsets, yg, err_flag, workspace,
                          stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().moe_grouped_down_gemm(ctypes.byref(p), _ptr(hg), _ptr(hg_scales), _ptr(w2), _ptr(w2_scales),
                                       _ptr(masked_m), _ptr(offsets), _ptr(yg), _ptr(err_flag), _ptr(workspace),
                                       nbytes, _stream(stream)), "moe_grouped_down_gemm")


def moe_grouped_ffn(p: Problem, xg, xg_scales, w13, w13_scales, w2, w2_scales, masked_m, offsets, hg, hg_scales, yg,
                    err_flag, workspace, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().moe_grouped_ffn(ctypes.byref(p), _ptr(xg), _ptr(xg_scales), _ptr(w13), _ptr(w13_scales), _ptr(w2),
                                 _ptr(w2_scales), _ptr(masked_m), _ptr(offsets), _ptr(hg), _ptr(hg_scales), _ptr(yg),
                                 _ptr(err_flag), _ptr(workspace), nbytes, _stream(stream)), "moe_grouped_ffn")


def moe_route_permute(p: Problem, logits, x, phys_to_log, ids, w, masked_m, offsets, row_of, src_of, xg, xg_scales,
                      err_flag, workspace, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().moe_route_permute(ctypes.byref(p), _ptr(logits), _ptr(x), _ptr(phys_to_log), _ptr(ids), _ptr(w),
                                   _ptr(masked_m), _ptr(offsets), _ptr(row_of), _ptr(src_of), _ptr(xg),
                                   _ptr(xg_scales), _ptr(err_flag), _ptr(workspace), nbytes, _stream(stream)),
           "moe_route_permute")


def moe_ffn_combine(p: Problem, xg, xg_scales, w13, w13_scales, w2, w2_scales, masked_m, offsets, row_of, w, hg,
                    hg_scales, yg, out, err_flag, workspace, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().moe_ffn_combine(ctypes.byref(p), _ptr(xg), _ptr(xg_scales), _ptr(w13), _ptr(w13_scales), _ptr(w2),
                                 _ptr(w2_scales), _ptr(masked_m), _ptr(offsets), _ptr(row_of), _ptr(w), _ptr(hg),
                                 _ptr(hg_scales), _ptr(yg), _ptr(out), _ptr(err_flag), _ptr(workspace), nbytes,
                                 _stream(stream)), "moe_ffn_combine")


def moe_combine(p: Problem, yg, row_of, w, out, stream=None) -> None:
    _check(lib().moe_combine(ctypes.byref(p), _ptr(yg), _ptr(row_of), _ptr(w), _ptr(out), _stream(stream)),
           "moe_combine")


def _mx_args(values, codes, scales, name: str):
    """dtype, rows, cols and addresses of an MXFP4 conversion; leading dimensions count as rows."""
    d, addr = _values(values, name)
    if values.dim() == 2:
        rows, cols = values.shape
        lead = (rows,)
    elif values.dim() > 0:
        *lead, cols = values.shape
        lead = tuple(lead)
        rows = torch.Size(lead).numel()
    else:
        raise ValueError("%s: expected rows of values" % name)
    if cols % 32:
        raise ValueError("%s: rows of %d values are not whole blocks of 32" % (name, cols))
    return (d, rows, cols, addr, _arg(codes, "codes", torch.uint8, (*lead, cols // 2)),
            _arg(scales, "scales", torch.uint8, (*lead, cols // 32)))


def moe_mx_quantize(x, codes, scales, stream=None) -> None:
    """x [..., cols] (float32 or bfloat16) -> MXFP4 codes [..., cols/2] and scale bytes [..., cols/32] (uint8)."""
    d, rows, cols, px, pc, ps = _mx_args(x, codes, scales, "x")
    _check(lib().moe_mx_quantize(d, rows, cols, px, pc, ps, _stream(stream)), "moe_mx_quantize")


def moe_mx_dequantize(codes, scales, out, stream=None) -> None:
    """MXFP4 codes and scale bytes -> the values they stand for, out [..., cols] (float32 or bfloat16)."""
    d, rows, cols, po, pc, ps = _mx_args(out, codes, scales, "out")
    _check(lib().moe_mx_dequantize(d, rows, cols, pc, ps, po, _stream(stream)), "moe_mx_dequantize")


def _nseq(p: Problem, seq_offsets) -> int:
    if seq_offsets is None:
        return 1
    if seq_offsets.dim() != 1 or seq_offsets.numel() < 2:
        raise ValueError("seq_offsets: expected the nseq + 1 offsets of nseq >= 1 segments")
    return seq_offsets.numel() - 1


def moe_balance_workspace_bytes(p: Problem, nseq: int = 1) -> int:
    return lib().moe_balance_workspace_bytes(ctypes.byref(p), nseq)


def moe_balance_loss(p: Problem, logits, ids, valid, seq_offsets, score: str, coef: float, loss, counts, prob_sum,
                     tokens, err_flag, workspace, stream=None) -> None:
    """Load-balance loss of the router per segment, with the per-expert counts and score sums (moe.h).
    valid: uint8 [T] or None; seq_offsets: int32 [nseq + 1] or None (one segment); score: "softmax" or "sigmoid"."""
    B, i32, f32 = _nseq(p, seq_offsets), torch.int32, torch.float32
    _check(lib().moe_balance_loss(
        ctypes.byref(p), _arg(logits, "logits", f32, (p.T, p.E)), _arg(ids, "ids", i32, (p.T, p.K)),
        _arg(valid, "valid", torch.uint8, (p.T,)), _arg(seq_offsets, "seq_offsets", i32, (B + 1,)), B, SCORES[score],
        coef, _arg(loss, "loss", f32, (B,)), _arg(counts, "counts", i32, (B, p.E)),
        _arg(prob_sum, "prob_sum", f32, (B, p.E)), _arg(tokens, "tokens", i32, (B,)), _ptr(err_flag),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)), "moe_balance_loss")


def moe_balance_loss_backward(p: Problem, logits, valid, seq_offsets, score: str, coef: float, counts, tokens, dloss,
                              dlogits, stream=None) -> None:
    """Gradient of moe_balance_loss with respect to the logits; counts and tokens as that call wrote them."""
    B, i32, f32 = _nseq(p, seq_offsets), torch.int32, torch.float32
    _check(lib().moe_balance_loss_backward(
        ctypes.byref(p), _arg(logits, "logits", f32, (p.T, p.E)), _arg(valid, "valid", torch.uint8, (p.T,)),
        _arg(seq_offsets, "seq_offsets", i32, (B + 1,)), B, SCORES[score], coef,
        _arg(counts, "counts", i32, (B, p.E)), _arg(tokens, "tokens", i32, (B,)), _arg(dloss, "dloss", f32, (B,)),
        _arg(dlogits, "dlogits", f32, (p.T, p.E)), _stream(stream)), "moe_balance_loss_backward")


def _norm_args(x, block, gate, w_post, w_pre):
    """Common arguments of the norm calls: their type and shapes, and (dtype, T, H, x, block, gate kind, gate, w_post,
    w_pre)."""
    d, addr = _values(x, "x")
    if x.dim() != 2:
        raise ValueError("x: expected [T, H]")
    TH = T, H = x.shape
    dt, one = x.dtype, (H,)
    kind = MOE_GATE_NONE
    if gate is not None:
        kind = MOE_GATE_TOKEN if gate.dim() == 2 else MOE_GATE_CHANNEL
    return dt, TH, (d, T, H, addr, _arg(block, "block", dt, TH), kind,
                    _arg(gate, "gate", dt, (T, 1) if kind == MOE_GATE_TOKEN else one),
                    _arg(w_post, "w_post", dt, one), _arg(w_pre, "w_pre", dt, one))


def moe_block_norm_workspace_bytes(T: int, H: int) -> int:
    return lib().moe_block_norm_workspace_bytes(T, H)


def moe_block_norm(x, block, gate, w_post, w_pre, res_scale: float, eps: float, y, xn, stream=None) -> None:
    """y = x + res_scale * gate * rms(block) * w_post, xn = rms(y) * w_pre (moe.h).  x, block, y, xn [T, H];
    w_post, w_pre [H]; gate None, [H] (a value a channel) or [T, 1] (a value a token); block None: y = x; w_pre and
    xn None: only y."""
    dt, TH, a = _norm_args(x, block, gate, w_post, w_pre)
    _check(lib().moe_block_norm(*a, res_scale, eps, _arg(y, "y", dt, TH), _arg(xn, "xn", dt, TH), _stream(stream)),
           "moe_block_norm")


def moe_block_norm_backward(x, block, gate, w_post, w_pre, res_scale: float, eps: float, dy, dxn, dx, dblock, dgate,
                            dw_post, dw_pre, workspace, stream=None) -> None:
    """Gradient of moe_block_norm from its inputs: dx, dblock like x; dgate like the gate, dw_post and dw_pre [H],
    all three float32 and each None where it is not wanted."""
    dt, TH, a = _norm_args(x, block, gate, w_post, w_pre)
    one, f32 = TH[1:], torch.float32
    _check(lib().moe_block_norm_backward(
        *a, res_scale, eps, _arg(dy, "dy", dt, TH), _arg(dxn, "dxn", dt, TH), _arg(dx, "dx", dt, TH),
        _arg(dblock, "dblock", dt, TH), _arg(dgate, "dgate", f32, () if gate is None else gate.shape),
        _arg(dw_post, "dw_post", f32, one), _arg(dw_pre, "dw_pre", f32, one), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)), "moe_block_norm_backward")


def moe_eplb_record(p: Problem, masked_m, pass_index: int, window: int, load_window, stream=None) -> None:
    _check(lib().moe_eplb_record(ctypes.byref(p), _ptr(masked_m), int(pass_index), int(window), _ptr(load_window),
                                 _stream(stream)), "moe_eplb_record")


def moe_eplb_rebalance(p: Problem, load_window, window: int, phys_to_log, logical_load, new_phys_to_log, err_flag,
                       stream=None) -> None:
    _check(lib().moe_eplb_rebalance(ctypes.byref(p), _ptr(load_window), int(window), _ptr(phys_to_log),
                                    _ptr(logical_load), _ptr(new_phys_to_log), _ptr(err_flag), _stream(stream)),
           "moe_eplb_rebalance")


def moe_selftest_bounded_wait(cycles: int, err_flag, stream=None) -> None:
    _check(lib().moe_selftest_bounded_wait(int(cycles), _ptr(err_flag), _stream(stream)), "moe_selftest_bounded_wait")


def moe_eplb_invert(p2l, E: int, R: int):
    """Host helper: (logical_to_physical [E,R], logical_replica_count [E], max replicas)."""
    import numpy as np
    p2l = np.ascontiguousarray(p2l, dtype=np.int32)
    l2p = np.empty((E, R), np.int32)
    rc = np.empty(E, np.int32)
    r = lib().moe_eplb_invert(p2l.size, E, p2l.ctypes.data, R, l2p.ctypes.data, rc.ctypes.data)
    if r < 0:
        raise MoeError(r, "moe_eplb_invert")
    return l2p, rc, r
