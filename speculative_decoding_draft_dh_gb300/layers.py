"""The layers around the candidate head as differentiable functions: the embedding of drafted tokens and the
layer norm of the hidden rows, for training them together with the head (``distill.distill_loss``).

``embedding`` is ``binding.embed`` with ``binding.embed_backward`` as its gradient, ``layer_norm`` is
``binding.layer_norm`` with ``binding.layer_norm_backward``; the library computes all of them.

Without gradients both may be captured into a CUDA graph.  A training step that is captured calls the four
functions of ``binding`` instead: the backward pass that autograd would replay synchronises with the streams on
which the leaves were used before, which a capture does not allow.

There are no forward-mode derivatives: a tensor with a tangent is refused.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import binding as dh


def _no_capture(name):
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{name} with gradients cannot be captured into a CUDA graph: use binding.{name} and "
                           f"binding.{name}_backward")


def _no_tangents(name, *tensors):
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError(f"{name} has no forward-mode derivative")


def _rows(t):
    """t [..., d] as rows whose elements are adjacent."""
    flat = t if t.dim() == 2 else t.reshape(-1, t.shape[-1])
    return flat if flat.stride(-1) == 1 or flat.shape[-1] <= 1 else flat.contiguous()


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, tokens, scale):
        ctx.save_for_backward(tokens)
        ctx.vocab, ctx.scale = table.shape[0], scale
        return dh.embed(table, tokens, scale=scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        _no_capture("embed")
        tokens, = ctx.saved_tensors
        return dh.embed_backward(_rows(grad), tokens, ctx.vocab, scale=ctx.scale), None, None


def embedding(table, tokens, *, scale=1.0):
    """scale * table[tokens] for tokens int32 of any shape, differentiable in the table [vocab, d]; padding (a token
    outside the vocabulary) has a row of zeros and no gradient.  Returns [*tokens.shape, d]."""
    if not table.is_cuda:
        raise ValueError("table must be a CUDA tensor")
    if table.dim() != 2:
        raise ValueError("table must be [vocab, d]")
    _no_tangents("embedding", table)
    flat = tokens.reshape(-1)
    if table.requires_grad and torch.is_grad_enabled():
        _no_capture("embed")
        rows = _Embedding.apply(table, flat, float(scale))
    else:
        rows = dh.embed(table.detach(), flat, scale=float(scale))
    return rows.reshape(*tokens.shape, table.shape[1])


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, stats = dh.layer_norm(x, weight, bias, eps=eps, with_stats=True)
        ctx.save_for_backward(x, weight, stats)
        ctx.param_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        _no_capture("layer_norm")
        x, weight, stats = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = dh.layer_norm_backward(_rows(grad), x, stats, weight, param_dtype=ctx.param_dtype,
                                            with_x=need[0], with_weight=need[1], with_bias=need[2])
        return dx, dw, db, None


def layer_norm(x, weight=None, bias=None, *, eps=1e-5):
    """Layer norm of x [..., d] over its last dimension, differentiable in x, weight and bias [d] (fp32 or x's
    dtype)."""
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    _no_tangents("layer_norm", x, weight, bias)
    flat = _rows(x)
    given = [t for t in (x, weight, bias) if t is not None]
    if torch.is_grad_enabled() and any(t.requires_grad for t in given):
        _no_capture("layer_norm")
        y = _LayerNorm.apply(flat, weight, bias, float(eps))
    else:
        y, _ = dh.layer_norm(flat.detach(), weight, bias, eps=float(eps))
    return y.reshape(x.shape)
