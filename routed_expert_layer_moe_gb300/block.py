"""The layer inside its transformer block: the norm before it, the router's loss, the layer, and the norm
after it with gate and residual, which also norms the input of the next block.

    block = MoeBlock(layer, w_pre, w_post, gate, w_next)
    xn = block.enter(x)                       # rms(x) * w_pre
    logits = xn.float() @ W_g                 # the router's product is the caller's
    y, xn_next = block.leave(x, logits)       # x + res_scale * gate * rms(layer(xn)) * w_post, rms(y) * w_next

With sigmoid scores and groups of experts the router's call comes between:

    block.layer.route_grouped(logits, n_group, topk_group, bias, scale=2.5)
    y, xn_next = block.leave(x, logits, routed=True)

The buffers of the forward calls and of the loss are allocated once and every call only enqueues kernels on the
stream, so a step is graph-capturable after a first eager one.  leave_backward() and enter_backward() return new
tensors, allocated on the stream of the call: a caller that uses them on another stream orders the two streams, and
calls record_stream on what it drops there, as with any tensor of another stream.

What one pass leaves for its gradients is overwritten by the next one: layer.out and layer.ids by any forward pass of
the layer (of another block on it too), the results of a method of the block by its next call.  Where another
pass comes between a forward and its gradients (micro-batches, two blocks on one layer), keep copies and hand
them in: ids to balance(), counts and tokens to balance_backward(), out to leave_backward().  Calls that use each
other's results are ordered by the caller if they run on different streams, and so are two calls of one method."""
from __future__ import annotations

import torch

from . import _lib as L


class MoeBlock:
    """A MoeLayer with its norms and the balance loss of its router.  w_pre, w_post, w_next [H], gate None, [H] or
    [T, 1], all of the activations' type; w_next None: no norm of the next block's input.  score, coef, nseq: the scores,
    the factor and the segments of the balance loss (moe.h); they choose no router, see leave()."""

    def __init__(self, layer, w_pre, w_post, gate=None, w_next=None, res_scale: float = 1.0, eps: float = 1e-6,
                 score: str = "softmax", coef: float = 0.01, nseq: int = 1):
        p, x = layer.p, layer.out
        self.layer, self.p = layer, p
        self.w_pre, self.w_post, self.gate, self.w_next = w_pre, w_post, gate, w_next
        self.res_scale, self.eps, self.score, self.coef = res_scale, eps, score, coef
        f32, i32 = dict(dtype=torch.float32, device=x.device), dict(dtype=torch.int32, device=x.device)
        self.xn, self.y = torch.empty_like(x), torch.empty_like(x)
        self.xn_next = None if w_next is None else torch.empty_like(x)
        self.loss, self.tokens = torch.empty(nseq, **f32), torch.empty(nseq, **i32)
        self.counts, self.prob_sum = torch.empty((nseq, p.E), **i32), torch.empty((nseq, p.E), **f32)
        self.dlogits = torch.empty((p.T, p.E), **f32)
        scratch = lambda n: torch.empty(n, dtype=torch.uint8, device=x.device)  # noqa: E731
        # one for each call that may run beside the others on a stream of its own
        self.ws_balance = scratch(L.moe_balance_workspace_bytes(p, nseq))
        self.ws_leave, self.ws_enter = (scratch(L.moe_block_norm_workspace_bytes(p.T, p.H)) for _ in range(2))

    # -- forward ----------------------------------------------------------------
    def enter(self, x, stream=None):
        """The norm before: rms(x) * w_pre, the layer's and the router's input."""
        L.moe_block_norm(x, None, None, None, self.w_pre, self.res_scale, self.eps, None, self.xn, stream)
        return self.xn

    def leave(self, x, logits, stream=None, routed=False):
        """The layer on enter()'s result, and the norm after it: (y, the next block's normed input or None).  The layer
        routes by softmax top-k of the logits; routed: it takes the ids and weights that it holds, of a routing
        that the caller made (layer.route_grouped, or any that writes layer.ids and layer.w)."""
        if routed:
            self.layer.permute(self.xn, stream)
            self.layer.ffn_combine(stream)
        else:
            self.layer.forward(self.xn, logits, stream, fused=True)
        L.moe_block_norm(x, self.layer.out, self.gate, self.w_post, self.w_next, self.res_scale, self.eps, self.y,
                         self.xn_next, stream)
        return self.y, self.xn_next

    # -- the router's loss ------------------------------------------------------
    def balance(self, logits, valid=None, seq_offsets=None, stream=None, ids=None):
        """Balance loss per segment of the routing that leave() made; counts and score sums in counts, prob_sum.
        ids: that routing, if it is not the layer's last one any more."""
        L.moe_balance_loss(self.p, logits, self.layer.ids if ids is None else ids, valid, seq_offsets, self.score,
                           self.coef, self.loss, self.counts, self.prob_sum, self.tokens, self.layer.err,
                           self.ws_balance, stream)
        return self.loss

    def balance_backward(self, logits, dloss, valid=None, seq_offsets=None, stream=None, counts=None, tokens=None):
        """Gradient of balance() with respect to the logits.  counts, tokens: as that call left them, if another one
        came since."""
        if (counts is None) != (tokens is None):
            raise ValueError("counts and tokens belong together")
        if counts is None:
            counts, tokens = self.counts, self.tokens
        L.moe_balance_loss_backward(self.p, logits, valid, seq_offsets, self.score, self.coef, counts, tokens, dloss,
                                    self.dlogits, stream)
        return self.dlogits

    # -- gradients of the norms -------------------------------------------------
    def leave_backward(self, x, dy, dxn_next, stream=None, out=None):
        """Gradients of leave()'s norm: of x, of the layer's output, of gate, w_post and w_next (fp32).  dxn_next is
        None without w_next.  out: the layer's output in that leave(), if it is not the layer's last one any more."""
        f32 = dict(dtype=torch.float32, device=x.device)
        with L._allocate_on(stream):
            dx, dout = torch.empty_like(x), torch.empty_like(x)
            dgate = None if self.gate is None else torch.empty(self.gate.shape, **f32)
            dw_post = torch.empty(self.w_post.shape, **f32)
            dw_next = None if self.w_next is None else torch.empty(self.w_next.shape, **f32)
        L.moe_block_norm_backward(x, self.layer.out if out is None else out, self.gate, self.w_post, self.w_next,
                                  self.res_scale, self.eps, dy, dxn_next, dx, dout, dgate, dw_post, dw_next,
                                  self.ws_leave, stream)
        return dx, dout, dgate, dw_post, dw_next

    def enter_backward(self, x, dxn, dy=None, stream=None):
        """Gradients of enter(): of x (plus dy, what else reaches x) and of w_pre (fp32)."""
        with L._allocate_on(stream):
            dx = torch.empty_like(x)
            dw_pre = torch.empty(self.w_pre.shape, dtype=torch.float32, device=x.device)
        L.moe_block_norm_backward(x, None, None, None, self.w_pre, self.res_scale, self.eps, dy, dxn, dx, None, None,
                                  None, dw_pre, self.ws_enter, stream)
        return dx, dw_pre
