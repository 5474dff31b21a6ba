"""A language model's head with what stands on either side of it: the embedding and the final norm before it, gradient
clipping after its backward, and penalties, biases, masks and sampling on its logits when it answers.

    python examples/head_step.py [--tokens N] [--hidden D] [--vocab V] [--steps K] [--requests B] [--answer M]
                                 [--tied] [--four-bits] [--temperature T] [--top-k K] [--top-p P] [--min-p P]

Trains a head on synthetic tokens for K steps (norm -> linear cross-entropy -> backward -> clip -> SGD; with --tied the
inputs are looked up in the head's own weight), then lets it answer B requests for M tokens (norm -> logits, with
--four-bits from a weight in 4 bits -> penalties, biases, mask -> the best token, or with --temperature a random one).
Inputs are random and seeded; no data or trained weights are involved.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import linear_cross_entropy_tmem_gb300 as flce  # noqa: E402


class Head(torch.nn.Module):
    """The final norm of a residual stream and the projection to the vocabulary."""

    def __init__(self, hidden: int, vocab: int, *, dtype=torch.bfloat16, seed: int = 0, eps: float = 1e-6):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.eps = eps
        self.norm = torch.nn.Parameter(torch.ones(hidden, dtype=dtype, device="cuda"))
        self.weight = torch.nn.Parameter(
            (torch.randn(vocab, hidden, generator=g, device="cuda") * hidden ** -0.5).to(dtype))

    def loss(self, x, residual, targets):
        """Mean cross-entropy of the next token, and the residual stream after x was added."""
        hidden, stream = flce.add_rms_norm(x, self.norm, residual, eps=self.eps)
        loss, _, _, _ = flce.linear_cross_entropy(hidden, self.weight, targets)
        return loss, stream

    def tied_loss(self, ids, residual, targets):
        """The same where x is looked up in the head's own weight, scaled by the width's square root."""
        x = flce.embedding(self.weight, ids, scale=self.weight.shape[1] ** 0.5)
        return self.loss(x, residual, targets)

    @torch.no_grad()
    def four_bits(self) -> flce.MxFp4:
        """The weight in 4 bits, for answers."""
        return flce.mxfp4_quantize(self.weight)

    @torch.no_grad()
    def answer(self, x, residual, *, weight4=None, **options):
        """Logits of the last position, processed for choosing a token (see ``process_logits``); ``weight4`` is
        :meth:`four_bits`'s."""
        hidden = flce.flce_add_rms_norm(x, self.norm, residual, eps=self.eps, need_rstd=False).y
        logits = hidden @ self.weight.t() if weight4 is None else flce.mxfp4_logits(hidden, weight4)
        return flce.process_logits(logits, **options)


def train_step(head: Head, x, residual, targets, *, lr: float, max_norm: float):
    """One step on hidden states x, or on tokens x (whole numbers) of a tied head; returns (loss, norm of the gradients
    before clipping)."""
    for p in head.parameters():
        p.grad = None
    loss, _ = head.loss(x, residual, targets) if x.is_floating_point() else head.tied_loss(x, residual, targets)
    loss.backward()
    grads = [p.grad for p in head.parameters()]
    norm = flce.clip_grad_norm_(grads, max_norm)
    with torch.no_grad():
        for p in head.parameters():
            p.sub_(p.grad, alpha=lr)
    return loss.detach(), norm


def decode(head: Head, embed, prompts, steps: int, *, repetition=1.2, presence=0.3, frequency=0.1, bias=None, mask=None,
           weight4=None, sampling=None, generator=None):
    """Answers [B, steps] to ``prompts`` [B, P]: greedy, or with ``sampling`` (options of ``sample_tokens``, numbers for
    all requests) random.  The stand-in for a model's layers is the embedding of the last token, added to a residual
    stream that keeps all before it."""
    b, n = prompts.shape
    tokens = torch.full((b, n + steps), -1, dtype=torch.int64, device="cuda")
    tokens[:, :n] = prompts
    lens = torch.full((b,), n, dtype=torch.int64, device="cuda")
    full = lambda x: torch.full((b,), float(x), device="cuda")  # noqa: E731
    options = dict(tokens=tokens, lens=lens, prompt_lens=lens.clone(), repetition=full(repetition),
                   presence=full(presence), frequency=full(frequency), mask=mask, weight4=weight4)
    if bias is not None:
        options["bias_ids"], options["bias"] = bias
    if sampling is not None:
        sampling = {k: full(x) if k != "top_k" else full(x).long() for k, x in sampling.items()}
    stream = flce.flce_embedding(embed, prompts[:, :-1].contiguous(), out_dtype=torch.float32).sum(1)
    last = prompts[:, -1].contiguous()
    for _ in range(steps):
        x = flce.flce_embedding(embed, last)
        answer = head.answer(x, stream, **options)
        last = answer.token
        if sampling is not None:
            uniform = torch.rand(b, generator=generator, device="cuda")
            last = flce.sample_tokens(answer.logits, uniform, **sampling).token
        stream = stream + x
        tokens.scatter_(1, lens[:, None], last[:, None])
        lens += 1
    return tokens[:, n:]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--answer", type=int, default=16)
    ap.add_argument("--tied", action="store_true")
    ap.add_argument("--four-bits", action="store_true")
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--top-k", type=int, default=0)
    ap.add_argument("--top-p", type=float, default=1.0)
    ap.add_argument("--min-p", type=float, default=0.0)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(1)
    head = Head(a.hidden, a.vocab)
    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    residual = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    targets = torch.randint(0, a.vocab, (a.tokens,), generator=g, device="cuda")
    if a.tied:
        x = torch.randint(0, a.vocab, (a.tokens,), generator=g, device="cuda")
    for k in range(a.steps):
        loss, norm = train_step(head, x, residual, targets, lr=2.0, max_norm=1.0)
        print(f"step {k}: loss {float(loss):.4f}, gradient norm {float(norm):.4f}")
    embed = torch.randn(a.vocab, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    if a.tied:
        embed = head.weight.detach()
    prompts = torch.randint(0, a.vocab, (a.requests, 12), generator=g, device="cuda")
    sampling = None
    if a.temperature > 0:
        sampling = dict(temperature=a.temperature, top_k=a.top_k, top_p=a.top_p, min_p=a.min_p)
    words = (a.vocab + 31) // 32
    mask = torch.full((a.requests, words), -1, dtype=torch.int32, device="cuda")
    mask[:, 0] = -2  # token 0 is never an answer
    for i, row in enumerate(decode(head, embed, prompts, a.answer, mask=mask, sampling=sampling, generator=g,
                                      weight4=head.four_bits() if a.four_bits else None).tolist()):
        print(f"request {i}: {row}")


if __name__ == "__main__":
    main()
