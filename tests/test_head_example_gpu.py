"""The operators on either side of the head used together, as examples/head_step.py uses them: a training step's
gradients against 64-bit autograd, clipping that holds, and answers that obey penalties, biases and masks."""
from __future__ import annotations

import pytest
import torch

import oracle
from examples.head_step import Head, decode, train_step

pytestmark = pytest.mark.gpu


def _inputs(n, d, v, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, d, generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn(n, d, generator=g, device="cuda").to(torch.bfloat16)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[::17] = -100
    return x, r, t


@pytest.mark.parametrize("n,d,v", [(300, 200, 1000), (512, 1280, 3000)])
def test_training_step_gradients(n, d, v):
    """Gradients of x, the residual, the norm and the head within the framework's bound for gradients (1e-2 relative
    Frobenius error) of the composition in 64 bits."""
    x, r, t = _inputs(n, d, v)
    head = Head(d, v)
    with torch.no_grad():
        head.norm.add_(0.1 * torch.randn_like(head.norm))
    lx, lr = x.clone().requires_grad_(True), r.clone().requires_grad_(True)
    loss, stream = head.loss(lx, lr, t)
    (loss + 1e-3 * stream.float().square().mean()).backward()
    ref = [a.detach().double().requires_grad_(True) for a in (x, r, head.norm, head.weight)]
    h = ref[0] + ref[1]
    y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * ref[2]
    want = torch.nn.functional.cross_entropy(y @ ref[3].t(), t, ignore_index=-100) + 1e-3 * h.square().mean()
    want.backward()
    assert abs(float(loss.detach()) + 1e-3 * float(stream.detach().double().square().mean()) - float(want.detach())) <= 4e-3
    for got, w in zip((lx.grad, lr.grad, head.norm.grad, head.weight.grad), ref):
        assert oracle.relative_frobenius(got.float().cpu(), w.grad.cpu()) <= 1e-2


def test_training_steps_clip_and_learn():
    x, r, t = _inputs(512, 256, 1000)
    head = Head(256, 1000)
    losses = []
    for _ in range(8):
        before = [p.detach().clone() for p in head.parameters()]
        loss, norm = train_step(head, x, r, t, lr=1.0, max_norm=0.05)
        losses.append(float(loss))
        step = torch.cat([(p.detach() - b).flatten().float() for p, b in zip(head.parameters(), before)])
        # gradients are rounded once after clipping (2^-8 of each), parameters once more (2^-8 of each)
        size = torch.cat([p.detach().flatten().float() for p in head.parameters()]).norm()
        assert float(norm) > 0.05 and float(step.norm()) <= 0.05 * (1 + 2.0 ** -7) + float(size) * 2.0 ** -8
    assert losses[-1] < losses[0]


def test_answers_obey_masks_biases_and_penalties():
    v, d, b = 3000, 256, 5
    head = Head(d, v)
    g = torch.Generator(device="cuda").manual_seed(7)
    embed = torch.randn(v, d, generator=g, device="cuda").to(torch.bfloat16)
    prompts = torch.randint(0, v, (b, 9), generator=g, device="cuda")
    mask = torch.zeros(b, (v + 31) // 32, dtype=torch.int32, device="cuda")
    mask[:, 10] = -1  # 32 words are allowed
    out = decode(head, embed, prompts, 12, mask=mask)
    assert torch.all((out >= 320) & (out < 352))
    # a frequency penalty above the logits' range: no word twice
    out = decode(head, embed, prompts, 20, mask=mask, frequency=1e4)
    assert all(len(set(row)) == 20 for row in out.tolist())
    # a large bias decides, and nothing allowed gives -1
    ids = torch.full((b, 1), 77, dtype=torch.int64, device="cuda")
    out = decode(head, embed, prompts, 3, bias=(ids, torch.full((b, 1), 1e6, device="cuda")), repetition=1.0)
    assert torch.all(out == 77)
    out = decode(head, embed, prompts, 1, mask=torch.zeros_like(mask))
    assert torch.all(out == -1)
