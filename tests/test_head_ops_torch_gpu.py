"""What the torch calls on either side of the head owe torch: counts of in-place changes, and the same results whether
the tensors are marshalled natively or in Python."""
from __future__ import annotations

import pytest
import torch

import linear_cross_entropy_tmem_gb300 as F
from linear_cross_entropy_tmem_gb300 import head_ops

pytestmark = pytest.mark.gpu

BF, SP = torch.bfloat16, torch.float32


@pytest.fixture(params=["native", "python"])
def path(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(head_ops, "_call", lambda *a: None)
    return request.param


def test_a_saved_tensor_that_a_call_wrote_raises_in_backward(path):
    z = torch.randn(3, 100, device="cuda", requires_grad=True)
    logits = z * 1.0
    loss = logits.exp().sum()  # saves its result
    used = logits.square().sum()  # saves logits
    F.process_logits(logits, out=logits)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        used.backward()
    loss.backward()  # its saved tensor was not written
    p = torch.randn(50, device="cuda", requires_grad=True)
    g = p * 2.0
    loss = g.square().sum()
    with torch.no_grad():
        F.clip_grad_norm_([g], 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_counts_of_in_place_changes(path):
    """One for what is written, none for what is read or for a tensor that the call made; a view's base counts with it;
    inference tensors, which keep no count, are taken."""
    z, out, flat = torch.randn(4, 64, device="cuda"), torch.empty(4, 64, device="cuda"), torch.empty(200, device="cuda")
    g = [torch.randn(10, 10, device="cuda"), torch.randn(7, device="cuda"), torch.empty(0, device="cuda")]
    all_of = lambda: [t._version for t in (z, out, flat, *g)]  # noqa: E731
    start = all_of()
    since = lambda: [a - b for a, b in zip(all_of(), start)]  # noqa: E731
    F.process_logits(z)
    F.grad_norm(g)
    assert since() == [0] * 6
    assert F.process_logits(z, out=out).logits is out
    assert since() == [0, 1, 0, 0, 0, 0]
    F.process_logits(z, out=z)
    assert since() == [1, 1, 0, 0, 0, 0]
    F.clip_grad_norm_(g, 1.0, outputs=[flat[:100].view(10, 10), flat[100:107], flat[:0]])
    assert since() == [1, 1, 3, 0, 0, 0]
    F.clip_grad_norm_(g, 1.0)
    assert since() == [1, 1, 3, 1, 1, 1]
    with torch.inference_mode():
        t = torch.randn(4, 64, device="cuda")
        F.process_logits(t, out=t)
        F.clip_grad_norm_([t], 1.0)


def test_what_the_loss_calls_write_counts_as_changed():
    h, w, b = (torch.randn(s, device="cuda").to(BF) for s in ((40, 64), (100, 64), (100,)))
    t = torch.randint(0, 100, (40,), device="cuda")
    f = F.flce_forward(h, w, t, b)
    outs = tuple(torch.empty_like(x) for x in (h, w, b))
    start = [x._version for x in (h, w, b, *outs)]
    got = F.flce_backward(h, w, t, f.lse, f.n_valid, torch.ones(1, device="cuda"), b, outputs=outs)
    assert all(a is o for a, o in zip(got, outs))
    assert [x._version - s for x, s in zip((h, w, b, *outs), start)] == [0, 0, 0, 1, 1, 1]
    F.scale_gradient(outs[0], torch.full((1,), 0.5, device="cuda"))
    assert outs[0]._version == start[3] + 2
    p = torch.randn(50, device="cuda", requires_grad=True)
    g = p * 2.0
    loss = g.square().sum()
    F.scale_gradient(g, torch.full((1,), 0.5, device="cuda"))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_second_derivatives_raise():
    h, w, nw = (torch.randn(s, device="cuda").to(BF).requires_grad_(True) for s in ((40, 64), (100, 64), (64,)))
    t = torch.randint(0, 100, (40,), device="cuda")
    for y in (F.add_rms_norm(h, nw), F.add_rms_norm(h, nw, h.detach())[0], F.linear_cross_entropy(h, w, t)[0],
              F.linear_cross_entropy(h, w, t, grad_in_forward=False)[0]):
        g, = torch.autograd.grad(y.float().sum(), h, create_graph=True)
        assert torch.isfinite(g.float()).all()
        with pytest.raises(RuntimeError, match="differentiable once"):
            (g.float().square().sum() + h.float().sum()).backward()
