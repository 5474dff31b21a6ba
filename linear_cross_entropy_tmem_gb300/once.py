"""Gradients that have no derivative of their own.

The library's backward calls return tensors without a graph.  Under ``create_graph=True`` such a gradient would pass
for a constant, and a loss of it would lose its part of the second derivative without a word.  (A decorator that looks
at the upstream gradient alone does not see that the gradient also depends on the inputs.)
"""
from __future__ import annotations

from typing import Optional

import torch


class _Once(torch.autograd.Function):
    """``grad`` as it is, tied to what it depends on by a backward that raises."""

    @staticmethod
    def forward(ctx, what, grad, *sources):
        ctx.what = what
        return grad

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"flce: {ctx.what} is differentiable once: its gradients have no derivative")


def once(what: str, grad: Optional[torch.Tensor], *sources: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """``grad``, which a backward of ``what`` computed from ``sources``; where a graph of the backward is being
    recorded, a second derivative through it raises."""
    if grad is None or not torch.is_grad_enabled() or not any(s is not None and s.requires_grad for s in sources):
        return grad
    return _Once.apply(what, grad, *sources)
