"""The five calls of the forward pass chained over caller-owned device buffers.

PyTorch provides device memory and the stream; each step runs in the
library's kernels.  Buffers are allocated once (static shapes), so a forward
call is graph-capturable after a first eager call."""
from __future__ import annotations

import torch

from . import _lib as L

TORCH_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8, "e2m1": torch.uint8,
               "mxfp4": torch.uint8}


class MoeLayer:
    """Buffers and calls for one problem.  Weights are slot-indexed tensors on the
    device: w13 [P+S, 2I, H], w2 [P+S, H, I] (e4m3: uint8 codes with fp32 block
    scales w13_s [P+S, 2I/128, H/128], w2_s [P+S, H/128, I/128]; e2m1: the same
    with two codes per byte, w13 [P+S, 2I, H/2], w2 [P+S, H, I/2]).  With e4m3
    or e2m1 weights the grouped activations xg, hg are e4m3 with 1x128 scales.
    mxfp4: uint8 codes, two to a byte, w13 [P+S, 2I, H/2], w2 [P+S, H, I/2], with a
    scale byte per 32 codes, w13_s [P+S, 2I, H/32], w2_s [P+S, H, I/32] (as
    moe_mx_quantize writes them); xg and hg have the same form.

    train (bf16 experts): the buffers of a training pass too.  forward(x, logits, save=True) keeps g and u of the
    experts in 8 bits, and backward(dout) gives the gradients of that pass.  What it reads (ids, w, row_of, masked_m,
    offsets, xg, yg, gu, gu_s) is overwritten by the layer's next forward pass, with or without save: where other
    passes come between a forward and its gradient (micro-batches), take a MoeLayer for each, on the same weights.
    backward() itself overwrites hg and its own buffers (dyg, wg, dgu, dxg, dw).  Those five hold nothing between calls:
    layers of one problem whose backward() calls follow each other on one stream can have them in common, by assigning one
    layer's to the others.

    saved: whether those buffers hold one pass whose g and u were kept; backward() refuses where they do not.  The
    layer's methods keep it up as they are called.  A replay of a captured graph calls none of them, nor does what a
    program writes into the buffers itself: one that calls backward() after such a pass sets saved = True first.  One
    that puts a checkpoint of its own in the place of gu answers for the other buffers too: saved is True from then on,
    until the next routing or dispatch."""

    def __init__(self, problem: L.Problem, act: str, wt: str, out: str, w13, w2, w13_s=None, w2_s=None,
                 phys_to_log=None, device="cuda", train=False):
        self.p = problem
        self.act, self.wt, self.out_dt = act, wt, out
        st = L.moe_check_problem(problem)
        if st != L.MOE_OK:
            raise L.MoeError(st, "problem")
        p = problem
        dev = torch.device(device)
        self.w13, self.w2, self.w13_s, self.w2_s = w13, w2, w13_s, w2_s
        self.p2l = phys_to_log
        S = p.has_shared
        rows = L.moe_grouped_rows(p)
        self.rows = rows
        i32 = dict(dtype=torch.int32, device=dev)
        self.ids = torch.empty((p.T, p.K), **i32)
        self.w = torch.empty((p.T, p.K), dtype=torch.float32, device=dev)
        self.masked_m = torch.empty(p.P + S, **i32)
        self.offsets = torch.empty(p.P + S + 1, **i32)
        self.row_of = torch.empty((p.T, p.K + S), **i32)
        self.src_of = torch.full((rows,), -1, **i32)
        f8, mx = wt in ("e4m3", "e2m1"), wt == "mxfp4"
        pack = 2 if mx else 1  # MXFP4: two codes a byte
        gd = TORCH_DTYPE[wt]
        yd = torch.float32 if wt == "f32" else torch.bfloat16
        self.xg = torch.empty((rows, p.H // pack), dtype=gd, device=dev)
        self.hg = torch.empty((rows, p.I // pack), dtype=gd, device=dev)
        self.yg = torch.empty((rows, p.H), dtype=yd, device=dev)
        group, sd = (32, torch.uint8) if mx else (128, torch.float32)
        self.xg_s = torch.empty((rows, p.H // group), dtype=sd, device=dev) if f8 or mx else None
        self.hg_s = torch.empty((rows, p.I // group), dtype=sd, device=dev) if f8 or mx else None
        self.out = torch.empty((p.T, p.H), dtype=TORCH_DTYPE[out], device=dev)
        self.err = torch.zeros(1, **i32)
        # routings and dispatches so far, and after how many of them hg, yg and gu were written from what these left
        self._pass, self._hg_of, self._yg_of, self._gu_of = 0, -1, -1, -1
        self.train = bool(train)
        if train:
            if wt != "bf16":
                raise L.MoeError(L.MOE_ERR_UNSUPPORTED, "training of %s experts" % wt)
            bf16 = dict(dtype=torch.bfloat16, device=dev)
            self._gu = torch.empty((rows, 2 * p.I), dtype=torch.uint8, device=dev)
            self.gu_s = torch.empty((rows, 2 * p.I // L.FP8_GROUP), dtype=torch.float32, device=dev)
            self.dyg = torch.empty((rows, p.H), **bf16)
            self.dxg = torch.empty((rows, p.H), dtype=torch.float32, device=dev)
            self.dgu = torch.empty((rows, 2 * p.I), **bf16)
            self.wg = torch.empty(rows, dtype=torch.float32, device=dev)
            self.dw = torch.empty((p.T, p.K), dtype=torch.float32, device=dev)
        nbytes = max(L.moe_workspace_bytes(p), 256)
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)

    @property
    def saved(self):
        return self._gu_of == self._yg_of == self._pass

    @saved.setter
    def saved(self, held):
        self._hg_of = -1
        self._gu_of = self._yg_of = self._pass if held else -1

    @property
    def gu(self):
        return self._gu

    @gu.setter
    def gu(self, codes):
        self._gu = codes
        self.saved = True

    # -- the steps --------------------------------------------------------------
    def route(self, logits, stream=None):
        self._pass += 1
        L.moe_route_topk(self.p, logits, self.ids, self.w, stream)

    def route_grouped(self, logits, n_group, topk_group, bias=None, renormalize=True, scale=1.0, stream=None):
        """DeepSeek-style grouped top-k (sigmoid, bias for the choice only) in place of route()."""
        self._pass += 1
        L.moe_route_grouped_topk(self.p, logits, bias, n_group, topk_group, self.ids, self.w,
                                 renormalize=renormalize, scale=scale, stream=stream)

    def permute(self, x, stream=None):
        self._pass += 1
        L.moe_permute(self.p, self.ids, x, self.p2l, self.masked_m, self.offsets, self.row_of, self.src_of,
                      self.xg, self.xg_s, self.err, self.ws, stream)

    def swiglu(self, stream=None):
        L.moe_grouped_swiglu_gemm(self.p, self.xg, self.xg_s, self.w13, self.w13_s, self.masked_m, self.offsets,
                                  self.hg, self.hg_s, self.err, self.ws, stream)
        self._hg_of = self._pass

    def swiglu_save(self, stream=None):
        """swiglu() that keeps g and u in 8 bits for backward(): gu, gu_s."""
        self._training("swiglu_save()")
        L.moe_grouped_swiglu_gemm_save(self.p, self.xg, self.w13, self.masked_m, self.offsets, self.hg, self.gu,
                                       self.gu_s, self.err, stream)
        self._hg_of = self._gu_of = self._pass

    def down(self, stream=None):
        L.moe_grouped_down_gemm(self.p, self.hg, self.hg_s, self.w2, self.w2_s, self.masked_m, self.offsets,
                                self.yg, self.err, self.ws, stream)
        self._yg_of = self._hg_of

    def ffn(self, stream=None):
        """gate/up + SwiGLU and down in one call (moe_grouped_ffn; one launch, but two for mxfp4 and f32); same outputs as
        swiglu() + down()."""
        L.moe_grouped_ffn(self.p, self.xg, self.xg_s, self.w13, self.w13_s, self.w2, self.w2_s, self.masked_m,
                          self.offsets, self.hg, self.hg_s, self.yg, self.err, self.ws, stream)
        self._hg_of = self._yg_of = self._pass

    def combine(self, stream=None):
        L.moe_combine(self.p, self.yg, self.row_of, self.w, self.out, stream)

    def route_permute(self, logits, x, stream=None):
        """route() + permute() in one call (moe_route_permute; one launch for small batches)."""
        self._pass += 1
        L.moe_route_permute(self.p, logits, x, self.p2l, self.ids, self.w, self.masked_m, self.offsets, self.row_of,
                            self.src_of, self.xg, self.xg_s, self.err, self.ws, stream)

    def ffn_combine(self, stream=None):
        """gate/up, down and combine in one call (moe_ffn_combine); same outputs as swiglu() + down() + combine()."""
        L.moe_ffn_combine(self.p, self.xg, self.xg_s, self.w13, self.w13_s, self.w2, self.w2_s, self.masked_m,
                          self.offsets, self.row_of, self.w, self.hg, self.hg_s, self.yg, self.out, self.err, self.ws,
                          stream)
        self._hg_of = self._yg_of = self._pass

    def forward(self, x, logits, stream=None, fused=False, save=False):
        """route -> permute -> gate/up -> down -> combine; returns self.out.  fused=True makes the
        same pass with the fused calls: route_permute() and ffn_combine().  save=True (a layer with train=True):
        gate/up keeps what backward() needs; route_permute() and ffn_save(), whatever fused is."""
        if save:
            self._training("forward(save=True)")
            self.route_permute(logits, x, stream)
            self.ffn_save(stream)
            return self.out
        if fused:
            self.route_permute(logits, x, stream)
            self.ffn_combine(stream)
            return self.out
        self.route(logits, stream)
        self.permute(x, stream)
        self.swiglu(stream)
        self.down(stream)
        self.combine(stream)
        return self.out

    # -- training ---------------------------------------------------------------
    def _training(self, what):
        if not self.train:
            raise ValueError("%s: the layer was made without train=True" % what)

    def ffn_save(self, stream=None):
        """ffn_combine() of a training pass: gate/up that keeps g and u, down, combine."""
        self.swiglu_save(stream)
        if self.rows:  # the down call takes no empty buffers
            self.down(stream)
        else:
            self._yg_of = self._hg_of
        self.combine(stream)

    def backward(self, dout, dw13=None, dw2=None, accumulate=False, weights=True, score="softmax", logits=None,
                 renormalize=True, scale=1.0, add=None, stream=None):
        """Gradients of the last forward pass, made with save=True, from dout, the gradient of its output: (dx, dlogits,
        dw13, dw2).  A ValueError where the layer holds no such pass (see saved).
        dw13, dw2: tensors for the weights' gradients, like w13 and w2 (bf16) or in float32; None: new ones like
        the weights; accumulate: added to the ones given (float32); weights=False: none, both are None.  score: the
        router of that pass, "softmax" (route) or "sigmoid" (route_grouped, with its logits, renormalize and scale).
        add [T, E]: added to dlogits, for instance the balance loss's gradient.  New tensors are allocated on the
        stream of the call."""
        self._training("backward()")
        if not self.saved:
            raise ValueError("backward(): the layer does not hold a pass made with save=True (see saved)")
        if accumulate and (not weights or dw13 is None or dw2 is None):
            raise ValueError("accumulate: expected dw13 and dw2 to add to")
        p = self.p
        with L._allocate_on(stream):
            dx = torch.empty_like(self.out)
            dlogits = torch.empty((p.T, p.E), dtype=torch.float32, device=self.out.device)
            if weights:
                dw13 = torch.empty_like(self.w13) if dw13 is None else dw13
                dw2 = torch.empty_like(self.w2) if dw2 is None else dw2
            else:
                dw13 = dw2 = None
        ptr = L._ptr  # the layer's own buffers, as in its other methods
        state = (ptr(self.yg), ptr(self.row_of), ptr(self.ids), ptr(self.w), ptr(self.xg), ptr(self.w13), ptr(self.w2),
                 ptr(self.gu), ptr(self.gu_s), ptr(self.masked_m), ptr(self.offsets))
        self._hg_of = -1  # hg holds h times the rows' weights from here on
        between = (ptr(self.dyg), ptr(self.wg), ptr(self.dgu), ptr(self.hg), ptr(self.dxg), ptr(self.dw))
        L._layer_backward(p, state, between, dout, dx, dlogits, dw13, dw2, self.err, score, logits, renormalize, scale, add,
                          accumulate, stream)
        return dx, dlogits, dw13, dw2
