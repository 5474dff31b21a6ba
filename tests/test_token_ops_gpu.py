"""GPU parity of the operators that lead from one token to the next (embedding and its gradient, 4-bit quantisation and
logits, sampling) against their formulas in 64 bits.

Tolerances.  u = 2^-24 is half a step of fp32; half a step of a stored type is ``finfo(t).eps / 2`` of the value.
  * A looked-up row is one fp32 product, rounded once: equal to torch's.
  * A row of the table's gradient sums n terms in fp32, in any order, and is scaled: within (n + 2) u of the sum of the
    terms' sizes, then rounded; added to what was there, one more fp32 step.
  * Codes and scales of 4 bits are whole numbers: equal.  Their values are powers of two times small integers: exact.
  * A product over blocks of 4-bit values: what a step of 64 columns adds is a multiple of 2^-2 of the smaller block's
    scale and the tensor core adds it to the fp32 sum, possibly cut off rather than rounded: within 2 u of the largest
    sum so far per step, at most the sum of the terms' sizes; bias and scale take 3 u more, the soft cap 2^-20 of its
    argument (the quotient, tanh of 2 units, the product).
  * Sampling: tokens and counts are equal.  (Weights are exact to 2^-31 and uniform numbers have 24 bits: of the cases
    here none lies that near a border.)  logprob: the quotient in 64 bits, a sum exact to 2^-30, one rounding.
"""
from __future__ import annotations

import math

import pytest
import torch

import linear_cross_entropy_tmem_gb300 as F

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, HF, SP = torch.bfloat16, torch.float16, torch.float32


def half_step(t, value):
    f = torch.finfo(t)
    return torch.clamp(value.abs() * (f.eps / 2), min=f.smallest_normal * f.eps / 2)


def within(got, want, tol, what):
    got, want = got.double(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    off = ((got - want).abs() - tol)[fine]
    assert off.numel() == 0 or float(off.max()) <= 0.0, (what, float(off.max()), int((off > 0).sum()), off.numel())


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(shape, t, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).to(t)


# ---------------------------------------------------------------------------------------------------
# Embedding
# ---------------------------------------------------------------------------------------------------
PAIRS = [(BF, BF), (HF, HF), (SP, SP), (BF, SP), (HF, SP)]


def skewed(n, v, seed, dtype=torch.int64):
    """Ids that crowd at the low end, some outside the table."""
    ids = (v * torch.rand(n, generator=gen(seed), device="cuda", dtype=torch.float64).pow(3)).long().clamp_(max=v - 1)
    ids[3::11] = -1
    ids[5::97] = v
    return ids.to(dtype)


def check_embedding(w, ids, scale, out_dtype):
    got = F.flce_embedding(w, ids, scale=scale, out_dtype=out_dtype)
    there = (ids >= 0) & (ids < w.shape[0])
    want = w[ids.long().clamp(0, w.shape[0] - 1)].float() * scale
    want = torch.where(there[..., None], want, torch.zeros_like(want)).to(out_dtype or w.dtype)
    assert got.shape == (*ids.shape, w.shape[1]) and got.dtype == want.dtype
    assert torch.equal(got, want)


@pytest.mark.parametrize("cols", [1, 7, 8, 64, 100, 257, 1283, 2048, 4096, 8200])
@pytest.mark.parametrize("types", PAIRS, ids=lambda t: f"{t[0]}-{t[1]}".replace("torch.", ""))
def test_embedding_forward(types, cols):
    t, o = types
    w = rand((301, cols), t, cols)
    for n, ids_t in ((1, torch.int64), (37, torch.int32), (5000, torch.int64)):
        check_embedding(w, skewed(n, 301, n, ids_t), math.sqrt(cols), o)
    check_embedding(w, skewed(24, 301, 3).view(2, 3, 4), 1.0, o)


def test_embedding_forward_views():
    wide = rand((50, 300), BF, 1)
    ids = skewed(40, 50, 2)
    check_embedding(wide[:, 8:8 + 128], ids, 1.0, None)    # rows apart, on 16-byte boundaries or not
    check_embedding(wide[:, 3:3 + 128], ids, 2.0, SP)
    check_embedding(wide[:1].expand(50, 300), ids, 1.0, None)
    check_embedding(rand((1, 16), SP, 3), torch.zeros(3, dtype=torch.int32, device="cuda"), 1.0, None)
    assert F.flce_embedding(wide, ids[:0]).shape == (0, 300)
    assert F.flce_embedding(wide, torch.tensor(7, device="cuda")).shape == (300,)
    special = torch.tensor([[float("nan"), float("inf"), -0.0, 1.0]], device="cuda")
    got = F.flce_embedding(special, torch.tensor([0, -1], device="cuda"))
    assert torch.isnan(got[0, 0]) and got[0, 1] == math.inf and torch.equal(got[1], torch.zeros(4, device="cuda"))
    for bad, err in ((dict(out_dtype=HF), F.token_ops.B.FlceError), (dict(scale=math.nan), F.token_ops.B.FlceError)):
        with pytest.raises(err):
            F.flce_embedding(wide, ids, **bad)
    with pytest.raises(TypeError, match="ids"):
        F.flce_embedding(wide, ids.float())
    with pytest.raises(ValueError, match="contiguous"):
        F.flce_embedding(wide, ids.view(2, 20).t())
    with pytest.raises(ValueError, match="adjacent"):
        F.flce_embedding(wide.t(), ids)


def bwd_ref(dout, ids, v, scale, pad=None, base=None):
    """The gradient in 64 bits and the sum of the sizes of each element's terms, and how many they are."""
    d = dout.shape[-1]
    ids, x = ids.reshape(-1).long(), dout.reshape(-1, d).double()
    on = (ids >= 0) & (ids < v)
    if pad is not None:
        on &= ids != pad
    dw = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, ids[on], x[on] * scale)
    size = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, ids[on], (x[on] * scale).abs())
    n = torch.bincount(ids[on], minlength=v)[:, None].double()
    if base is not None:
        dw, size = dw + base.double(), size + base.double().abs()
    return dw, size, n


def check_backward(dout, ids, v, t, scale=1.0, pad=None, base=None):
    want, size, n = bwd_ref(dout, ids, v, scale, pad, base)
    got = F.flce_embedding_backward(dout, ids, v, scale=scale, padding_idx=pad, dtype=t,
                                    dweight=None if base is None else base.clone())
    assert got.dtype == t and got.shape == (v, dout.shape[-1])
    within(got, want, half_step(t, want) + (n + 4) * U * 1.0001 * size, "dweight")
    if base is None:
        assert torch.all(got[(n == 0).squeeze(1)] == 0)
    else:
        assert torch.equal(got[(n == 0).squeeze(1)], base[(n == 0).squeeze(1)])
    return got


@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 64, 500, 4096, 4097, 9001])
@pytest.mark.parametrize("v,cols", [(1, 8), (5, 100), (300, 257), (1023, 64), (1024, 130), (70001, 24)])
def test_embedding_backward(n, v, cols):
    ids = skewed(n, v, n + v)
    dout = rand((n, cols), SP, n + cols)
    check_backward(dout, ids, v, SP, scale=3.5)
    if n in (33, 4097):
        base = rand((v, cols), SP, 5)
        check_backward(dout, ids, v, SP, scale=0.5, base=base)
        check_backward(dout, ids.to(torch.int32), v, SP, pad=0)


@pytest.mark.parametrize("types", PAIRS, ids=lambda t: f"{t[0]}-{t[1]}".replace("torch.", ""))
@pytest.mark.parametrize("cols", [64, 77, 2048, 2056, 4099])
def test_embedding_backward_types(types, cols):
    t, o = types
    ids = skewed(700, 200, cols)
    dout = rand((700, cols), o, cols)
    check_backward(dout, ids, 200, t, scale=math.sqrt(cols), pad=1)
    check_backward(dout, ids, 200, t, base=rand((200, cols), t, 9, 4.0))


def test_embedding_backward_runs():
    """One id for all tokens, runs that end on the borders of a block's tokens, tables of a million rows."""
    d = 40
    for n in (64, 320, 5000, 70000):
        dout = rand((n, d), SP, n)
        check_backward(dout, torch.full((n,), 3, device="cuda"), 7, SP)
        check_backward(dout, torch.arange(n, device="cuda") // 32, n, SP)
        check_backward(dout, torch.arange(n, device="cuda") // 48, n // 3, BF)
        check_backward(dout, torch.full((n,), -5, device="cuda"), 7, SP)
    check_backward(rand((1000, 8), BF, 1), torch.randint(0, 1 << 20, (1000,), generator=gen(1), device="cuda"), 1 << 20, BF)
    ids = torch.randint(0, 1 << 21, (3000,), generator=gen(2), device="cuda")
    check_backward(rand((3000, 8), HF, 1), ids, (1 << 21) + 1, HF)


def test_embedding_backward_views_and_repeats():
    n, v, d = 900, 50, 96
    ids = skewed(n, v, 1).view(3, 300)
    wide = rand((n, 200), BF, 2)
    a = check_backward(wide[:, 8:8 + d], ids.view(-1), v, BF)
    check_backward(wide[:, 3:3 + d], ids.view(-1), v, BF)
    check_backward(wide[:1, :d].expand(n, d), ids.view(-1), v, BF)
    # a wider table's columns: what stands beside them stays
    table = rand((v, 2 * d), BF, 3)
    kept = table.clone()
    F.flce_embedding_backward(wide[:, 8:8 + d], ids.view(-1), v, dweight=table[:, :d])
    assert torch.equal(table[:, d:], kept[:, d:])
    want, size, m = bwd_ref(wide[:, 8:8 + d], ids, v, 1.0, base=kept[:, :d])
    within(table[:, :d], want, half_step(BF, want) + (m + 4) * U * size, "dweight")
    # the same bits every time, and in a caller's workspace
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(a, F.flce_embedding_backward(wide[:, 8:8 + d], ids.view(-1), v, workspace=ws))
    with pytest.raises(ValueError, match="workspace"):
        F.flce_embedding_backward(wide[:, :d], ids.view(-1), v, workspace=ws[:64])
    with pytest.raises(ValueError, match="shape"):
        F.flce_embedding_backward(wide[:, :d], ids, v)
    with pytest.raises(ValueError, match="dweight"):
        F.flce_embedding_backward(wide[:, :d], ids.view(-1), v, dweight=table)
    # NaN and infinity stay in the rows that have them
    x = rand((64, 8), SP, 4)
    x[10, 3], x[11, 4] = math.nan, math.inf
    i = torch.arange(64, device="cuda")
    got = F.flce_embedding_backward(x, i, 64)
    assert torch.equal(torch.isnan(got), torch.isnan(x)) and got[11, 4] == math.inf


def test_embedding_autograd():
    v, d = 100, 64
    w = rand((v, d), BF, 1).requires_grad_(True)
    ids = skewed(60, v, 2).view(3, 20)
    out = F.embedding(w, ids, scale=8.0, padding_idx=2, out_dtype=SP)
    up = rand(out.shape, SP, 3)
    (out * up).sum().backward()
    want, size, n = bwd_ref(up, ids, v, 8.0, 2)
    within(w.grad, want, half_step(BF, want) + (n + 4) * U * size, "grad")
    w.grad = None
    F.embedding(w, ids).sum().backward()  # an expanded upstream gradient
    assert torch.equal(w.grad[:, 0].double(), torch.bincount(ids[(ids >= 0) & (ids < v)], minlength=v).double())
    w.grad = None
    g, = torch.autograd.grad(F.embedding(w, ids).square().sum(), w, create_graph=True)
    with pytest.raises(RuntimeError, match="once"):
        g.sum().backward()
    # differences of the looked-up sum along a direction
    ww = rand((v, d), SP, 4).requires_grad_(True)
    out = F.embedding(ww, ids, scale=2.0)
    (out.double().sin().sum()).backward()
    step = rand((v, d), SP, 5)
    f = lambda x: float(F.flce_embedding(x, ids, scale=2.0).double().sin().sum())  # noqa: E731
    h = 2.0 ** -10
    slope = (f(ww.detach() + h * step) - f(ww.detach() - h * step)) / (2 * h)
    # third derivatives of sin(2 x) are at most 8: h^2 / 6 * 8 |step|^3 for each term, and fp32's rounding of 2 x over h
    terms = step[ids.clamp(0, v - 1)].abs().double()
    tol = float((h * h / 6 * 8 * terms.pow(3)).sum()) + terms.numel() ** 0.5 * 16 * U / h * 4
    assert abs(slope - float((ww.grad.double() * step.double()).sum())) <= tol


# ---------------------------------------------------------------------------------------------------
# 4 bits
# ---------------------------------------------------------------------------------------------------
GRID = [0, .5, 1, 1.5, 2, 3, 4, 6]


def mx_ref(x):
    """Codes [n, blocks * 32] and exponents + 127 [n, blocks], by the borders between the grid's values."""
    n, d = x.shape
    b = -(-d // 32)
    x = torch.nn.functional.pad(x.double(), (0, b * 32 - d)).view(n, b, 32)
    top = x.abs().amax(2)
    k = torch.where(top > 0, torch.frexp(top).exponent.double() - 3, -127.0).clamp(-127, 125)
    bad = ~torch.isfinite(x).all(2)
    k = torch.where(bad, torch.zeros_like(k), k)
    a = x.abs() / torch.exp2(k)[..., None]
    low = torch.tensor([.25, 1.25, 2.5, 5], dtype=torch.float64, device=x.device)
    high = torch.tensor([.75, 1.75, 3.5], dtype=torch.float64, device=x.device)
    code = torch.bucketize(a, low) + torch.bucketize(a, high, right=True) + 8 * torch.signbit(x).long()
    code = torch.where(bad[..., None], torch.zeros_like(code), code)
    return code.view(n, b * 32), torch.where(bad, 255, (k + 127).long())


def mx_values(code, e):
    grid = torch.tensor(GRID + [-g for g in GRID], dtype=torch.float64, device=code.device)
    scale = torch.where(e == 255, math.nan, torch.exp2(e.double() - 127))
    return (grid[code].view(*e.shape, 32) * scale[..., None]).view(code.shape)


def tiled(e):
    n, b = e.shape
    nt, kt = -(-n // 128), -(-b // 4)
    e = torch.nn.functional.pad(e, (0, kt * 4 - b, 0, nt * 128 - n)).to(torch.uint8)
    return e.view(nt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous()


def check_quantize(x):
    q = F.mxfp4_quantize(x)
    code, e = mx_ref(x.reshape(-1, x.shape[-1]))
    pairs = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    assert torch.equal(q.codes, pairs)
    assert torch.equal(q.scales, tiled(e))
    want = mx_values(code, e)[:, :x.shape[-1]]
    for t in (SP, BF, HF):
        got = F.mxfp4_dequantize(q, t)
        assert got.dtype == t and got.shape == want.shape
        assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want.to(t), nan=7.0))
    return q, want


@pytest.mark.parametrize("t", [BF, HF, SP], ids=str)
@pytest.mark.parametrize("n,d", [(1, 1), (1, 4096), (3, 31), (5, 32), (7, 33), (127, 128), (128, 136), (129, 160),
                                 (33, 255), (2, 256), (40, 257), (300, 1283), (260, 2048), (1, 16384)])
def test_mxfp4_quantize(t, n, d):
    check_quantize(rand((n, d), t, n * 7 + d) * torch.exp(rand((d,), SP, 1)).to(t))


def test_mxfp4_every_border():
    """The grid's values, the borders between them and their neighbours in fp32, in both signs, at several scales."""
    g = torch.tensor(GRID, dtype=torch.float64)
    at = torch.cat([g, (g[1:] + g[:-1]) / 2, torch.tensor([5.0, 6.5, 7.0, 7.99])])
    at = torch.cat([at, torch.nextafter(at.float(), torch.tensor(9.0)).double(),
                    torch.nextafter(at.float(), torch.tensor(-9.0)).double().clamp(min=0)])
    at = torch.cat([at, -at])
    for power in (-140, -127, -126, -60, 0, 3, 90, 125):
        x = torch.zeros(at.numel(), 32, dtype=torch.float64)
        x[:, 0], x[:, 1] = 4.0, at  # the block's largest is 4 to 8 units
        x[:, 17] = -at / 2
        check_quantize((x * 2.0 ** power).clamp(-3.4e38, 3.4e38).float().cuda())
    sub = torch.tensor([1e-45, 2e-40, 1.1754944e-38, -1e-39], device="cuda").repeat(8)[None]
    check_quantize(sub)


def test_mxfp4_special_values_and_views():
    x = rand((6, 96), SP, 1)
    x[0, 3], x[1, 40], x[2, 95], x[3, 0:32] = math.nan, math.inf, -math.inf, 0.0
    x[4, 5] = -0.0
    check_quantize(x)
    wide = rand((50, 400), BF, 2)
    check_quantize(wide[:, 8:8 + 128])
    check_quantize(wide[:, 3:3 + 128])
    check_quantize(wide[:1].expand(9, 400))
    check_quantize(rand((2, 3, 64), HF, 3))
    q = F.mxfp4_quantize(wide[:0])
    assert q.shape == (0, 400) and F.mxfp4_dequantize(q).shape == (0, 400)
    q = F.mxfp4_quantize(wide)
    for bad in (F.MxFp4(q.codes[:, :-16], q.scales, 400), F.MxFp4(q.codes, q.scales[:, :1], 400),
                F.MxFp4(q.codes, q.scales, 300), F.MxFp4(q.codes.float(), q.scales, 400), F.MxFp4(q.codes, q.scales, 0)):
        with pytest.raises(ValueError, match="codes"):
            F.mxfp4_dequantize(bad)


def check_logits(h, w, bias=None, scale=1.0, cap=0.0, out_dtype=None, **kw):
    q = F.mxfp4_quantize(w)
    got = F.mxfp4_logits(h, q, bias, logit_scale=scale, softcap=cap, out_dtype=out_dtype, **kw)
    hv = mx_values(*mx_ref(h.reshape(-1, h.shape[-1])))[:, :h.shape[-1]]
    wv = F.mxfp4_dequantize(q).double()
    z, size = hv @ wv.t(), hv.abs() @ wv.abs().t()
    tol = (2 * math.ceil(h.shape[-1] / 64) + 2) * U * size
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    z, tol = z * scale, tol * abs(scale) + 3 * U * size * abs(scale)
    if cap:
        tol = tol + 2.0 ** -20 * z.abs().clamp(max=cap)
        z = cap * torch.tanh(z / cap)
    t = out_dtype or h.dtype
    assert got.dtype == t and got.shape == (*h.shape[:-1], w.shape[0])
    within(got.view(z.shape) if got.is_contiguous() else got, z, half_step(t, z) * 1.01 + tol, "logits")
    return got


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 100, 128, 129, 208, 209, 417])
@pytest.mark.parametrize("v,d", [(1000, 64), (129, 96), (260, 4096), (2048, 320)])
def test_mxfp4_logits(n, v, d):
    h, w = rand((n, d), BF, n + d), rand((v, d), BF, v)
    check_logits(h, w, out_dtype=SP)


@pytest.mark.parametrize("d", [1, 31, 32, 33, 64, 65, 128, 192, 193, 255, 256, 257, 511, 513, 1283, 8192])
def test_mxfp4_logits_widths(d):
    h, w = rand((37, d), SP, d), rand((700, d), HF, d + 1)
    check_logits(h, w, out_dtype=SP)


@pytest.mark.parametrize("o", [BF, HF, SP], ids=str)
@pytest.mark.parametrize("t", [BF, HF, SP], ids=str)
def test_mxfp4_logits_epilogue(t, o):
    h, w = rand((70, 320), t, 1), rand((1003, 320), t, 2, 0.3)
    for bt in (BF, HF, SP):
        check_logits(h, w, rand((1003,), bt, 3), 0.7, 0.0, o)
    check_logits(h, w, rand((1003,), t, 3), 0.5, 5.0, o)
    check_logits(h, w, None, -1.5, 30.0, o)


def test_mxfp4_logits_many_tiles():
    """More tiles than SMs, so that blocks take several: one token, and two tiles of tokens."""
    w = rand((50000, 256), BF, 1)
    check_logits(rand((1, 256), BF, 2), w)
    check_logits(rand((300, 256), BF, 3), w, rand((50000,), BF, 4), 1.0, 20.0, SP)


def test_mxfp4_logits_views_special_values_and_repeats():
    w = rand((500, 128), BF, 1)
    wide = rand((40, 300), BF, 2)
    check_logits(wide[:, 8:8 + 128], w)
    check_logits(wide[:, 3:3 + 128], w)
    check_logits(rand((2, 5, 128), BF, 3), w)
    check_logits(rand((128,), BF, 4), w)
    q = F.mxfp4_quantize(w)
    h = rand((40, 128), BF, 5)
    want = F.mxfp4_logits(h, q)
    # into rows of a wider matrix, what stands beside them stays
    big = torch.full((41, 700), 5.0, dtype=BF, device="cuda")
    got = F.mxfp4_logits(h, q, out=big[:40, 100:600])
    assert got.data_ptr() == big[:, 100:].data_ptr() and torch.equal(big[:40, 100:600], want)
    assert torch.all(big[:, :100] == 5) and torch.all(big[:, 600:] == 5) and torch.all(big[40] == 5)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")  # scales that would be NaN
    for _ in range(3):
        assert torch.equal(want, F.mxfp4_logits(h, q, workspace=ws))
    assert F.flce_read_device_status(ws) == 0
    assert F.mxfp4_logits(h[:0], q).shape == (0, 500)
    # a NaN block of one token or one entry stays there
    h2 = h.clone()
    h2[3, 70] = math.inf
    w2 = w.clone()
    w2[130, 5] = math.nan
    bad = F.mxfp4_logits(h2, F.mxfp4_quantize(w2))
    nan = torch.zeros_like(bad, dtype=torch.bool)
    nan[3], nan[:, 130] = True, True
    assert torch.equal(torch.isnan(bad), nan)
    assert torch.equal(bad[~nan], want[~nan])
    for f in (lambda: F.mxfp4_logits(h[:, :96], q), lambda: F.mxfp4_logits(h, q, torch.zeros(499, device="cuda")),
              lambda: F.mxfp4_logits(h, q, out=big), lambda: F.mxfp4_logits(h, q, workspace=ws[:1000])):
        with pytest.raises(ValueError):
            f()


# ---------------------------------------------------------------------------------------------------
# Sampling
# ---------------------------------------------------------------------------------------------------
def sample_ref(z, u, t=None, k=None, p=None, m=None):
    """Token, log-probability and count of one row, from its definition in 64 bits."""
    z = z.double()
    nan = torch.isnan(z)
    if nan.any():
        return int(nan.nonzero()[0]), math.nan, 1
    n = int((z > -math.inf).sum())
    if n == 0:
        return -1, -math.inf, 0
    t = 1.0 if t is None else float(t)
    by = torch.argsort(z, descending=True, stable=True)[:n]
    if not t > 0:
        return int(by[0]), 0.0, 1
    if k is not None and 0 < int(k) < z.numel():
        by = by[:int(k)]
    top = z[by[0]]
    w = (z[by] == math.inf).double() if top == math.inf else torch.exp((z[by] - top) / t)
    keep = torch.ones_like(w, dtype=torch.bool)
    if p is not None and float(p) < 1:
        keep[1:] &= w.cumsum(0)[:-1] < float(p) * w.sum()
    if m is not None and float(m) > 0:
        keep &= w >= min(float(m), 1.0)
    by, w = by[keep], w[keep]
    order = torch.argsort(by)
    by, w = by[order], w[order]
    u = min(max(float(u), 0.0), 1 - 2.0 ** -53) if u == u else 0.0
    upto = w.cumsum(0)
    some = torch.nonzero(w > 0).squeeze(1)
    at = min(int((upto <= u * upto[-1]).sum()), int(some[-1]))
    return int(by[at]), float(torch.log(w[at] / upto[-1])), len(by)


def check_sample(z, u=None, t=None, k=None, p=None, m=None, seed=0):
    b = z.shape[0]
    vec = lambda x, dt: None if x is None else torch.as_tensor(x, dtype=dt).expand(b).contiguous().cuda()  # noqa: E731
    u = torch.rand(b, generator=gen(seed + 99), device="cuda") if u is None else vec(u, SP)
    t, k, p, m = vec(t, SP), vec(k, torch.int64), vec(p, SP), vec(m, SP)
    r = F.sample_tokens(z, u, temperature=t, top_k=k, top_p=p, min_p=m)
    got = list(zip(r.token.tolist(), r.logprob.tolist(), r.kept.tolist()))
    at = lambda x, i: None if x is None else x[i].cpu()  # noqa: E731
    for i in range(b):
        tok, lp, n = sample_ref(z[i].cpu(), u[i].cpu(), at(t, i), at(k, i), at(p, i), at(m, i))
        what = (i, got[i], (tok, lp, n), at(t, i), at(k, i), at(p, i), at(m, i), float(u[i]))
        assert got[i][0] == tok and got[i][2] == n, what
        if math.isfinite(lp):
            assert abs(got[i][1] - lp) <= abs(lp) * 2 * U + 2.0 ** -29, what
        else:
            assert got[i][1] == lp or (math.isnan(lp) and math.isnan(got[i][1])), what
    return r


def logits(b, v, t, seed, scale=3.0):
    z = torch.randn(b, v, generator=gen(seed), device="cuda") * scale
    z[:, ::17] = -math.inf
    return z.to(t)


VOCABS = [1, 2, 31, 100, 1000, 2049, 8200, 32003, 151936]
FILTERS = [dict(), dict(t=0.7), dict(k=1), dict(k=50, t=0.8), dict(p=0.9), dict(m=0.05), dict(t=0.0),
           dict(k=40, p=0.95, m=0.02, t=1.3), dict(k=700, p=0.5), dict(p=0.999, t=2.0), dict(p=0.0), dict(m=1.0),
           dict(k=10 ** 9, p=1.0, m=0.0, t=1.0), dict(k=3000)]


@pytest.mark.parametrize("kw", FILTERS, ids=str)
@pytest.mark.parametrize("v", VOCABS)
def test_sample(v, kw):
    t = (SP, BF, HF)[v % 3]
    check_sample(logits(5, v, t, v), seed=v, **kw)


@pytest.mark.parametrize("t", [SP, BF, HF], ids=str)
def test_sample_settings_of_each_row(t):
    b, v = 40, 20011
    pick = lambda *x: torch.tensor(x)[torch.randint(0, len(x), (b,))]  # noqa: E731
    torch.manual_seed(5)
    z = logits(b, v, t, 1)
    z[7] = -math.inf
    z[9, 1:] = -math.inf
    check_sample(z, t=pick(0.0, 0.5, 1.0, 1.5), k=pick(0, 1, 5, 100, 5000), p=pick(1.0, 0.3, 0.9, 0.99),
                 m=pick(0.0, 0.01, 0.2))


def test_sample_ties():
    """Equal logits: the lowest indexes are kept, and share the mass alike."""
    for v in (64, 5000, 40000):
        z = torch.zeros(6, v, device="cuda")
        u = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.999, 1.0])
        check_sample(z, u)
        check_sample(z, u, k=v // 3)
        check_sample(z, u, p=0.25)
        check_sample(z, u, k=16, p=0.5)
        check_sample(z, u, m=1.0)
        z[:, 1::2] = 1.0
        z[:, 5::8] = -2.0
        check_sample(z.to(BF), u, k=v // 4 + 3)
        check_sample(z.to(BF), u, p=0.9)
        check_sample(z, u, p=0.9, k=v - v // 8)
    # -0 and +0 are one value
    z = torch.tensor([[0.0, -0.0, 0.0, -1.0, -0.0]], device="cuda")
    check_sample(z, 0.9, k=2)
    check_sample(z, 0.9, k=4)


def test_sample_special_values():
    inf = math.inf
    rows = torch.tensor([
        [1.0, inf, 2.0, inf, -inf, inf, 0.0, 5.0],
        [1.0, math.nan, 2.0, inf, -inf, math.nan, 0.0, 5.0],
        [-inf] * 8,
        [-3e38, -inf, -3.1e38, -3e38, -inf, -3.4e38, -3e38, -inf],
        [3.4e38, 3e38, -3.4e38, 3.4e38, 0.0, -inf, 1.0, 2.0],
        [-1e-30, 1e-30, 0.0, -0.0, 1e-38, -1e-38, 1e-45, -inf],
        [-inf, -inf, -inf, -inf, -inf, -5.0, -inf, -inf]], device="cuda")
    for kw in (dict(), dict(t=0.0), dict(k=2), dict(p=0.5), dict(m=0.5), dict(t=1e-6), dict(t=1e-45, k=3), dict(t=1e30),
               dict(t=inf), dict(t=-1.0), dict(t=math.nan), dict(p=math.nan), dict(m=math.nan), dict(m=7.0),
               dict(p=-1.0), dict(k=-3)):
        for u in (0.0, 0.3, 0.7, 1.0 - U):
            check_sample(rows, u, **kw)
    for u in (-1.0, 2.0, math.nan, inf):
        check_sample(rows, u)
        check_sample(rows, u, k=2)


def test_sample_views_and_repeats():
    wide = logits(9, 5003, BF, 4)
    for z in (wide[:, 8:4104], wide[:, 3:4100], wide[:1].expand(4, 5003), wide[::2]):
        check_sample(z, p=0.9, t=0.8)
        check_sample(z, k=33)
    z, u = logits(70, 30000, SP, 6), torch.rand(70, generator=gen(7), device="cuda")
    p = torch.full((70,), 0.97, device="cuda")
    a = F.sample_tokens(z, u, top_p=p)
    for _ in range(3):
        b = F.sample_tokens(z, u, top_p=p)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    e = F.sample_tokens(z[:0], u[:0])
    assert e.token.shape == (0,)
    for f in (lambda: F.sample_tokens(z, u[:3]), lambda: F.sample_tokens(z, u.double()),
              lambda: F.sample_tokens(z, u, top_k=torch.ones(70, device="cuda", dtype=torch.int32)),
              lambda: F.sample_tokens(z[0], u), lambda: F.sample_tokens(z.t(), u)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        F.sample_tokens(z.double(), u)


def test_sample_large_vocabularies():
    for v, t in ((262144, SP), (1 << 20, BF), (1 << 20, SP), ((1 << 20) - 3, SP)):
        z = logits(2, v, t, v)
        check_sample(z, p=0.9, seed=1)
        check_sample(z, k=20000, p=0.99, seed=2)
        check_sample(z, seed=3)


def test_sample_follows_the_distribution():
    """Evenly spaced uniform numbers choose each entry as often as its probability says, within one."""
    v, b = 50, 4096
    z = rand((v,), SP, 8, 2.0)
    u = (torch.arange(b, device="cuda") + 0.5) / b
    r = F.sample_tokens(z.expand(b, v), u, top_k=torch.full((b,), 20, device="cuda"))
    keep = torch.topk(z, 20).indices
    q = torch.zeros(v, dtype=torch.float64, device="cuda")
    q[keep] = torch.softmax(z[keep].double(), 0)
    count = torch.bincount(r.token, minlength=v).double()
    assert float((count - q * b).abs().max()) <= 1.0
