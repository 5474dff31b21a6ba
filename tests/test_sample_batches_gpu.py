"""Sampling from batches that are larger than the GPU's clusters: one CTA then holds a whole row, and a single step of its
histograms can hold all of the row's entries (equal logits, rows of two or three values).

Tolerances.  A weight below 2^-6 of the largest is 2^31 2^(-j / 32), at least 2^30, times 1 + q in whole units: the table
is cut by 1 unit, q (at most 2^-6) carries fp32's rounding of its argument, 0.7 units, its own, 1, and that of the product,
1 and 0.5, and the last bit is set, 1: 5.2 units, below 2^-27 of the weight.  (2^-35 above 2^-6.)  So are their sums, and
a quotient of two sums is within 2^-26, or 2^-34; in fp64 sums of 2^20 entries are within 2^-33, quotients 2^-32.  Every
input is checked to keep 2^-25, or 2^-31, of the mass between the sums and the borders (p and u of the whole), so that
tokens and counts have to be equal.  logprob: 2^-26 for the whole, and one rounding of the result and one of its logarithm.
"""
from __future__ import annotations

import pytest
import torch

import linear_cross_entropy_tmem_gb300 as F

from .test_token_ops_gpu import BF, HF, SP, U, sample_ref

pytestmark = pytest.mark.gpu

MARGIN = 2.0 ** -25, 2.0 ** -31  # with weights below 2^-6 of the largest, without


def clear_of_borders(z, u, k, p):
    """Whether no sum of weights comes near a border of the choice (all in 64 bits, T = 1, no min-p)."""
    z = z.double()
    by = torch.argsort(z, descending=True, stable=True)[:k or z.numel()]
    w = torch.exp(z[by] - z[by[0]])
    upto = w.cumsum(0)
    assert float(w[-1]) > 2.0 ** -11  # (a unit is less than 2^-30 of it)
    margin = MARGIN[float(w[-1]) >= 2.0 ** -6]
    if p < 1 and float((upto / upto[-1] - p).abs().min()) < margin:
        return False
    keep = upto - w < p * upto[-1] if p < 1 else torch.ones_like(w, dtype=torch.bool)
    by, order = by[keep].sort()
    upto = w[keep][order].cumsum(0)
    return float((upto / upto[-1] - u).abs().min()) >= margin


def around(z, part):
    """top-p one and a half entries before and behind the place where the values equal to the ``part``-th largest value
    end, as fp32."""
    z = z.double()
    values = torch.unique(z).flip(0)
    w = torch.exp(z - values[0])
    upto = float(w[z >= values[part]].sum())
    here = float(torch.exp(values[part] - values[0]))
    behind = float(torch.exp(values[min(part + 1, len(values) - 1)] - values[0]))
    whole = float(w.sum())
    return [float(torch.tensor(x, dtype=torch.float32)) for x in ((upto - 1.5 * here) / whole, (upto + 1.5 * behind) / whole)]


def rows_of(v, t):
    """(logits, top_k, top_p) of rows with a great many equal entries."""
    g = torch.Generator().manual_seed(v)
    one = lambda low: torch.full((v,), low).index_fill(0, torch.tensor([v // 3]), 0.0)  # noqa: E731
    out = [(one(-1.0), 0, 0.9999), (one(-1.0), 0, 0.5), (one(-7.0), 0, 0.9), (one(-7.0), 0, 0.95), (one(-7.3), 0, 0.9),
           (torch.zeros(v), 0, 0.9999), (torch.zeros(v), 0, 0.9996), (torch.zeros(v), v - 1000, 0.9996),
           (one(-1.0), v - v // 5, 0.9999), (one(-1.0), v - 3, 1.0)]
    two = torch.where(torch.rand(v, generator=g) < 0.5, 0.0, -0.5)
    three = 100 + 0.5 * torch.randint(-1, 2, (v,), generator=g)  # 16-bit logits with an offset
    out += [(two, 0, p) for part in (0, 1) for p in around(two, part)[:2 - part]]
    out += [(three, 0, p) for part in (0, 1, 2) for p in around(three.to(t).float(), part)[:2 - part // 2]]
    out += [(three, v - v // 7, 0.97), (two, v // 2 + v // 5, 0.8)]
    # other values close behind many equal ones
    near = torch.where(torch.rand(v, generator=g) < 0.75, -1.0, -1.0 - 0.004 * torch.rand(v, generator=g))
    out += [(near, 0, 0.9), (near, 0, 0.7), (near, v - v // 10, 0.9999)]
    return [(z.to(t), k, p) for z, k, p in out]


SHAPES = [(256, 262144, SP), (150, 262144, BF), (100, 151936, SP), (100, 151936, HF), (100, 1 << 20, BF)]


def inputs(v, t):
    rows = rows_of(v, t)
    g = torch.Generator().manual_seed(v + 1)
    u = []
    for z, k, p in rows:
        for _ in range(200):
            x = torch.rand((), generator=g)
            if clear_of_borders(z, float(x), k, p):
                break
        u.append(x)
    return rows, torch.stack(u)


@pytest.mark.parametrize("b,v,t", SHAPES, ids=str)
def test_many_equal_logits_in_a_large_batch(b, v, t):
    rows, u = inputs(v, t)
    n = len(rows)
    assert all(clear_of_borders(z, float(x), k, p) for (z, k, p), x in zip(rows, u))
    at = torch.arange(b) % n
    z = torch.stack([r[0] for r in rows]).cuda()[at.cuda()]
    k = torch.tensor([r[1] for r in rows])[at].cuda()
    p = torch.tensor([r[2] for r in rows], dtype=SP)[at].cuda()
    uu = u[at].cuda()
    r = F.sample_tokens(z, uu, top_k=k, top_p=p)
    wrong = []
    for i in range(n):
        tok, lp, kept = sample_ref(rows[i][0], u[i], None, torch.tensor(rows[i][1]), p[i].cpu())
        got = int(r.token[i]), int(r.kept[i])
        if got != (tok, kept) or not abs(float(r.logprob[i]) - lp) <= abs(lp) * 2 * U + 2.0 ** -26:
            wrong.append((i, rows[i][1:], got, float(r.logprob[i]), (tok, kept, lp)))
    assert not wrong, wrong
    # the same row anywhere in the batch, and by itself (in more CTAs): the same bits
    for a in r:
        assert torch.equal(a, a[:n][at.cuda()])
    for i in range(n):
        alone = F.sample_tokens(z[i:i + 1], uu[i:i + 1], top_k=k[i:i + 1], top_p=p[i:i + 1])
        assert all(torch.equal(x, y[i:i + 1]) for x, y in zip(alone, r)), (i, alone, [y[i] for y in r])
