"""A transformer's MLP block whose backward pass runs from 8-bit checkpoints.

    out = x + W2 f(W1 layernorm(x) + b1) + b2

What the block keeps between the passes is one 8-bit checkpoint each of the layer norm's
input and output and of the activation's input and output, and two floats per row: about
2.1 (width + hidden) bytes per token where the tensors themselves in 16 bits take
4 (width + hidden).  Frozen parameters and a forward pass without gradients keep less, down to nothing.  The layer norm,
the activation and the two weight-gradient calls are the library's kernels (gc_train.h); the plain products with W1 and
W2 are torch's.

Parameters are float32 (what the compressors and the optimizer work on) and are cast to
the input's type for the products.  Their gradients come out in float32, in memory of their own; with ``.grad`` preset to
views of a flat bucket, autograd adds them into the bucket that the compressors take (a caller of
:func:`~.train.linear_wgrad` can have the kernel add into the bucket itself).
"""
from __future__ import annotations

import math

import torch

from .train import act_backward, act_forward, layernorm_backward, layernorm_forward, linear_wgrad

__all__ = ["MlpBlock8", "mlp_block8"]


class _MlpBlock(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, ln_w, ln_b, w1, b1, w2, b2, kind, eps, grad):
        dt = x.dtype
        # what the backward pass will read: nothing without one, and nothing for frozen parameters only
        need = ctx.needs_input_grad
        first, second, third = (grad and any(need[i:j]) for i, j in ((0, 3), (3, 5), (5, 7)))
        n, mean, rstd, x_ck, n_ck = layernorm_forward(x, ln_w, ln_b, eps, pack_x=first, pack_y=second)
        h = torch.addmm(b1.to(dt), n, w1.to(dt).t())
        a, h_ck, a_ck = act_forward(h, kind, pack_x=first or second, pack_y=third)
        out = torch.addmm(b2.to(dt), a, w2.to(dt).t()).add_(x)
        none = (None, None)
        ctx.save_for_backward(ln_w, w1, w2, mean, rstd, *(x_ck or none), *(n_ck or none), *(h_ck or none), *(a_ck or none))
        ctx.kind = kind
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out):
        ln_w, w1, w2, mean, rstd, xc, xe, nc, ne, hc, he, ac, ae = ctx.saved_tensors
        need = ctx.needs_input_grad
        dt = d_out.dtype
        d_out = d_out.contiguous()
        grads = [None] * 10
        if need[5] or need[6]:
            grads[5:7] = linear_wgrad(d_out, ac, ae, w2.shape[1], bias=need[6])
        if any(need[:5]):
            d_h = act_backward(torch.mm(d_out, w2.to(dt)), ctx.kind, ckpt=(hc, he))
            if need[3] or need[4]:
                grads[3:5] = linear_wgrad(d_h, nc, ne, w1.shape[1], bias=need[4])
            if any(need[:3]):
                d_x, *grads[1:3] = layernorm_backward(torch.mm(d_h, w1.to(dt)), mean, rstd, ln_w, ckpt=(xc, xe))
                grads[0] = d_x.add_(d_out)
        return tuple(grads)


def mlp_block8(x, ln_w, ln_b, w1, b1, w2, b2, kind="gelu", eps=1e-5):
    """The block as a function; x [..., width] in float32, float16 or bfloat16 and of any strides, parameters float32."""
    for name, p in (("ln_w", ln_w), ("ln_b", ln_b), ("w1", w1), ("b1", b1), ("w2", w2), ("b2", b2)):
        if p.dtype != torch.float32:
            raise ValueError(f"{name} must be float32, got {p.dtype}")
    rows = x.reshape(-1, x.shape[-1])           # a view where there is one, of any strides
    if (rows.shape[1] > 1 and rows.stride(1) != 1) or (rows.shape[0] > 1 and rows.stride(0) < rows.shape[1]):
        rows = rows.contiguous()                 # the kernels take consecutive columns and rows that do not overlap
    return _MlpBlock.apply(rows, ln_w, ln_b, w1, b1, w2, b2, kind, eps, torch.is_grad_enabled()).view(x.shape)


class MlpBlock8(torch.nn.Module):
    """Module form of :func:`mlp_block8`."""

    def __init__(self, width, hidden, kind="gelu", eps=1e-5, device=None):
        super().__init__()
        kw = dict(dtype=torch.float32, device=device)
        self.kind, self.eps = kind, eps
        self.ln_w = torch.nn.Parameter(torch.ones(width, **kw))
        self.ln_b = torch.nn.Parameter(torch.zeros(width, **kw))
        self.w1 = torch.nn.Parameter(torch.empty(hidden, width, **kw).normal_(0, 1 / math.sqrt(width)))
        self.b1 = torch.nn.Parameter(torch.zeros(hidden, **kw))
        self.w2 = torch.nn.Parameter(torch.empty(width, hidden, **kw).normal_(0, 1 / math.sqrt(hidden)))
        self.b2 = torch.nn.Parameter(torch.zeros(width, **kw))

    def forward(self, x):
        return mlp_block8(x, self.ln_w, self.ln_b, self.w1, self.b1, self.w2, self.b2, self.kind, self.eps)
