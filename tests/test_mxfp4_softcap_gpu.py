"""The soft cap of the 4-bit logits at the ends of its range."""
from __future__ import annotations

import pytest
import torch

import linear_cross_entropy_tmem_gb300 as F

from .test_token_ops_gpu import BF, SP, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("cap", [1e-45, 1e-40, 2.9e-39, 1e-38, 1e-30])
def test_smallest_soft_caps(n, cap):
    """cap * tanh(z / cap) is 0 for z = 0, and the cap in z's sign for a z of ordinary size: tanh is 1 there within three
    units of 2^-24, and the product is rounded once, by 2^-24 of itself or by half a step of subnormal numbers."""
    h = rand((n, 96), BF, 1)
    h[1] = 0
    q = F.mxfp4_quantize(rand((300, 96), BF, 2))
    z = F.mxfp4_logits(h, q, out_dtype=SP)
    got = F.mxfp4_logits(h, q, softcap=cap, out_dtype=SP)
    cap = torch.tensor(cap, dtype=SP, device="cuda")
    large = z.abs() > 1e-20
    assert torch.all(z[1] == 0) and int(large.sum()) > 0.9 * 300 * (n - 1)
    assert torch.equal(got[z == 0], z[z == 0])
    want = torch.copysign(cap.expand_as(z), z)
    tol = float(cap) * 4 * 2.0 ** -24 + 2.0 ** -150
    assert torch.all((got.double() - want.double()).abs()[large] <= tol)
