"""What the autograd functions promise, on the CPU: the library's calls are stood in for by the same formulas in torch
(without a graph, as the library's results are), so that the classes themselves run."""
from __future__ import annotations

import pytest
import torch

from linear_cross_entropy_tmem_gb300 import api, head_ops


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


# ---------------------------------------------------------------------------------------------------
# The loss
# ---------------------------------------------------------------------------------------------------
def _loss_backward(hidden, weight, targets, lse, n_valid, dloss, bias=None, *, reduction="mean", frozen_head=False, **_):
    z = hidden @ weight.t() + (bias if bias is not None else 0.0)
    d = (torch.softmax(z, 1) - torch.nn.functional.one_hot(targets, weight.shape[0])) * dloss.reshape(-1, 1)
    d = d / len(targets) if reduction == "mean" else d
    if frozen_head:
        return d @ weight, None, None
    return d @ weight, d.t() @ hidden, d.sum(0) if bias is not None else None


def _loss_forward(hidden, weight, targets, bias=None, *, reduction="mean", **_):
    z = hidden @ weight.t() + (bias if bias is not None else 0.0)
    one, n = torch.zeros((), dtype=torch.int64), torch.tensor(len(targets))
    loss = torch.nn.functional.cross_entropy(z, targets, reduction=reduction)
    return api.ForwardResult(loss, torch.logsumexp(z, 1), one, n, torch.zeros(()), None, None)


def _loss_forward_backward(hidden, weight, targets, dloss, bias=None, *, frozen_head=False, **kw):
    f = _loss_forward(hidden, weight, targets, bias, **kw)
    return f, _loss_backward(hidden, weight, targets, f.lse, f.n_valid, dloss, bias, frozen_head=frozen_head, **kw)


@pytest.fixture
def loss_stand_ins(monkeypatch):
    monkeypatch.setattr(api, "flce_forward", torch.no_grad()(_loss_forward))
    monkeypatch.setattr(api, "flce_backward", torch.no_grad()(_loss_backward))
    monkeypatch.setattr(api, "flce_forward_backward", torch.no_grad()(_loss_forward_backward))
    monkeypatch.setattr(api, "scale_gradient", torch.no_grad()(lambda x, s: x.mul_(s)))


def _loss_leaves(bias, n=4, d=6, v=5):
    g = torch.Generator().manual_seed(2)
    leaves = [torch.randn(s, generator=g, dtype=torch.float64).requires_grad_(True) for s in ((n, d), (v, d), (v,))]
    return leaves[0], leaves[1], leaves[2] if bias else None, torch.randint(0, v, (n,), generator=g)


@pytest.mark.parametrize("in_forward,reduction", [(True, "mean"), (True, "sum"), (False, "mean"), (True, "none")])
@pytest.mark.parametrize("bias", [True, False])
def test_loss_second_derivatives_are_refused(loss_stand_ins, bias, in_forward, reduction):
    h, w, b, t = _loss_leaves(bias)
    f = lambda *a: api.linear_cross_entropy(a[0], a[1], t, a[2] if bias else None, reduction=reduction,  # noqa: E731
                                            grad_in_forward=in_forward)[0]
    leaves = (h, w, b) if bias else (h, w)
    assert torch.autograd.gradcheck(f, leaves)
    for of in leaves:
        g, = torch.autograd.grad(f(*leaves).sum(), of, create_graph=True)
        with pytest.raises(RuntimeError, match="differentiable once"):
            (g.square().sum() + h.sum()).backward()


def test_loss_gradients_that_are_constants(loss_stand_ins):
    """A backward without create_graph ties nothing, and a frozen head's gradient is refused all the same."""
    h, w, b, t = _loss_leaves(True)
    api.linear_cross_entropy(h, w, t, b)[0].backward()
    assert all(x.grad.grad_fn is None and not x.grad.requires_grad for x in (h, w, b))
    g, = torch.autograd.grad(api.linear_cross_entropy(h, w.detach(), t)[0], h, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        (g.square().sum() + h.sum()).backward()
