"""Training the candidate head: the distillation loss as a differentiable function.

The teacher's entries are what ``binding.draft_head`` (or any top-K of a target's logits) returns:
candidate ids and their exact logits.  The student's logits are the low-rank head's scores over the
whole vocabulary.  ``distill_loss`` is ``binding.distill_topk`` with ``binding.distill_topk_backward``
as its gradient; the library computes both.

A training step that is captured into a CUDA graph calls ``binding.distill_topk_step`` instead: the
backward pass that autograd would replay synchronises with the streams on which the leaves were
used before, which a capture does not allow.
"""
from __future__ import annotations

import torch

from . import binding as dh


def _no_capture():
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError("distill_loss cannot be captured into a CUDA graph: use binding.distill_topk_step")


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, idx, teacher, n_valid, temperature):
        loss, stats = dh.distill_topk(logits, idx, teacher, n_valid=n_valid, temperature=temperature)
        ctx.save_for_backward(logits, idx, teacher, n_valid, stats)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss):
        _no_capture()
        logits, idx, teacher, n_valid, stats = ctx.saved_tensors
        grad = dh.distill_topk_backward(logits, idx, teacher, stats, grad_loss.float().contiguous(), n_valid=n_valid,
                                        temperature=ctx.temperature)
        return grad, None, None, None, None


def distill_loss(logits, idx, teacher, *, n_valid=None, temperature=1.0):
    """Per-row loss of the student's logits [..., vocab] against the teacher's entries idx int32 and
    teacher fp32 [..., K] (n_valid int32 [...]), differentiable in the logits only: the teacher is a
    constant.  Returns fp32 [...]."""
    lead = logits.shape[:-1]
    if idx.shape[:-1] != lead or teacher.shape != idx.shape or (n_valid is not None and n_valid.shape != lead):
        raise ValueError("idx and teacher must be [..., K] and n_valid [...] over the logits' rows")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    _no_capture()
    flat = logits if logits.dim() == 2 else logits.reshape(-1, logits.shape[-1])
    loss = _Distill.apply(flat, idx.reshape(-1, idx.shape[-1]), teacher.detach().reshape(-1, teacher.shape[-1]),
                          None if n_valid is None else n_valid.reshape(-1), float(temperature))
    return loss.reshape(lead)
