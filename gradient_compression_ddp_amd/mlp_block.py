"""A transformer's MLP block whose backward pass runs from 8-bit checkpoints.

    out = x + W2 f(W1 layernorm(x) + b1) + b2

What the block keeps between the passes is one 8-bit checkpoint each of the layer norm's
input and output and of the activation's input and output, and two floats per row: about
2.1 (width + hidden) bytes per token where the tensors themselves in 16 bits take
4 (width + hidden).  The layer norm, the activation and the three weight-gradient calls are
the library's kernels (gc_train.h); the plain products with W1 and W2 are torch's.

Parameters are float32 (what the compressors and the optimizer work on) and are cast to
the input's type for the products.  Their gradients come out in float32; with ``.grad`` preset to
views of a flat bucket, autograd adds into the bucket that the compressors take.
"""
from __future__ import annotations

import math

import torch

from .train import act_backward, act_forward, layernorm_backward, layernorm_forward, linear_wgrad

__all__ = ["MlpBlock8", "mlp_block8"]


class _MlpBlock(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, ln_w, ln_b, w1, b1, w2, b2, kind, eps):
        dt = x.dtype
        n, mean, rstd, x_ck, n_ck = layernorm_forward(x, ln_w, ln_b, eps, pack_x=True, pack_y=True)
        h = torch.addmm(b1.to(dt), n, w1.to(dt).t())
        a, h_ck, a_ck = act_forward(h, kind, pack_x=True, pack_y=True)
        out = torch.addmm(b2.to(dt), a, w2.to(dt).t()).add_(x)
        ctx.save_for_backward(ln_w, w1, w2, mean, rstd, *x_ck, *n_ck, *h_ck, *a_ck)
        ctx.kind = kind
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out):
        ln_w, w1, w2, mean, rstd, xc, xe, nc, ne, hc, he, ac, ae = ctx.saved_tensors
        dt = d_out.dtype
        d_out = d_out.contiguous()
        d_w2, d_b2 = linear_wgrad(d_out, ac, ae, w2.shape[1])
        d_h = act_backward(torch.mm(d_out, w2.to(dt)), ctx.kind, ckpt=(hc, he))
        d_w1, d_b1 = linear_wgrad(d_h, nc, ne, w1.shape[1])
        d_x, d_lw, d_lb = layernorm_backward(torch.mm(d_h, w1.to(dt)), mean, rstd, ln_w, ckpt=(xc, xe))
        return d_x.add_(d_out), d_lw, d_lb, d_w1, d_b1, d_w2, d_b2, None, None


def mlp_block8(x, ln_w, ln_b, w1, b1, w2, b2, kind="gelu", eps=1e-5):
    """The block as a function; x [..., width] in float32, float16 or bfloat16 and of any strides, parameters float32."""
    for name, p in (("ln_w", ln_w), ("ln_b", ln_b), ("w1", w1), ("b1", b1), ("w2", w2), ("b2", b2)):
        if p.dtype != torch.float32:
            raise ValueError(f"{name} must be float32, got {p.dtype}")
    rows = x.reshape(-1, x.shape[-1])           # a view where there is one, of any strides
    if (rows.shape[1] > 1 and rows.stride(1) != 1) or (rows.shape[0] > 1 and rows.stride(0) < rows.shape[1]):
        rows = rows.contiguous()                 # the kernels take consecutive columns and rows that do not overlap
    return _MlpBlock.apply(rows, ln_w, ln_b, w1, b1, w2, b2, kind, eps).view(x.shape)


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
