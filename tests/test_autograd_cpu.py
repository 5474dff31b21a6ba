"""What the autograd functions promise, on the CPU: the library's calls are stood in for by the same formulas in torch
(without a graph, as the library's results are), so that the classes themselves run."""
from __future__ import annotations

import pytest
import torch

from linear_cross_entropy_tmem_gb300 import head_ops


def _norm_forward(x, weight=None, residual=None, *, eps, weight_offset, need_rstd):
    h = x if residual is None else x + residual
    rstd = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
    return head_ops.AddRmsNormResult(h * rstd * (weight + weight_offset), h, rstd.flatten() if need_rstd else None)


def _norm_backward(dy, h, rstd, weight, *, dh, weight_offset, need_dx, need_dresidual, need_dweight):
    g, n = dy * (weight + weight_offset), h * rstd[:, None]
    d = rstd[:, None] * (g - n * (g * n).mean(1, keepdim=True))
    d = d if dh is None else d + dh
    return head_ops.AddRmsNormGrads(d if need_dx else None, d if need_dresidual else None,
                                    (dy * n).sum(0) if need_dweight else None)


@pytest.fixture
def norm_stand_ins(monkeypatch):
    monkeypatch.setattr(head_ops, "flce_add_rms_norm", torch.no_grad()(_norm_forward))
    monkeypatch.setattr(head_ops, "flce_add_rms_norm_backward", torch.no_grad()(_norm_backward))


def _leaves(n=3, d=8):
    g = torch.Generator().manual_seed(1)
    return [torch.randn(s, generator=g, dtype=torch.float64).requires_grad_(True) for s in ((n, d), (d,), (n, d))]


@pytest.mark.parametrize("residual", [True, False])
def test_norm_first_derivatives(norm_stand_ins, residual):
    x, w, r = _leaves()
    if residual:
        assert torch.autograd.gradcheck(lambda *a: head_ops.add_rms_norm(*a, weight_offset=1.0), (x, w, r))
    else:
        assert torch.autograd.gradcheck(lambda *a: head_ops.add_rms_norm(*a), (x, w))


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("of", [0, 1])
def test_norm_second_derivatives_are_refused(norm_stand_ins, residual, of):
    """The backward's results have no graph: a loss of them must not pass for one that has (its other branch here has)."""
    x, w, r = _leaves()
    y = head_ops.add_rms_norm(x, w, r)[0] if residual else head_ops.add_rms_norm(x, w)
    u = torch.linspace(-1.0, 1.0, 8, dtype=torch.float64)
    g, = torch.autograd.grad((y * u).sum(), (x, w)[of], create_graph=True)  # the gradient itself may be had
    with pytest.raises(RuntimeError, match="differentiable once"):
        (g.square().sum() + x.sum()).backward()


def test_norm_gradients_that_are_constants(norm_stand_ins):
    """Where only the weight has a gradient, dweight does not depend on it: nothing to refuse.  And a backward without
    create_graph ties nothing."""
    x, w, r = _leaves()
    y, _ = head_ops.add_rms_norm(x.detach(), w, r.detach())
    g, = torch.autograd.grad(y.sum(), w, create_graph=True)
    assert not g.requires_grad
    y, h = head_ops.add_rms_norm(x, w, r)
    (y.sum() + h.sum()).backward()
    assert all(t.grad.grad_fn is None and not t.grad.requires_grad for t in (x, w, r))
