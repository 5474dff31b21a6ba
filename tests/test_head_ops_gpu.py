"""GPU parity of the operators on either side of the head (norm, gradient clipping, logit processing) against
their formulas in 64 bits.

Tolerances.  u = 2^-24 is half a step of fp32; half a step of the stored type is ``finfo(t).eps / 2`` of the
value (its smallest subnormal / 2 near zero).
  * A mean of squares over D columns adds positive terms in chains of at most a few hundred and a short tree,
    so rstd (its inverse root: half the error) and y = h rstd w are within 2^-17 relative in fp32.
  * The backward's value d = rstd (g - n c) + dh is within 2^-17 of the sum of its terms' sizes.
  * A column sum over N rows is within (N + 64) u of the sum of its terms' sizes, in any order.
  * The norm of the gradients sums fp32 groups of 8 in fp64: within 2^-20.
  * A processed logit takes at most five fp32 steps: within 8 u of the largest value on the way.
  * lse: chains of a few hundred positive terms and hardware exponentials (2 units of 2^-23): within 2^-16
    absolute plus 2^-22 of its size.
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
    """Half a step of type t at `value` (64-bit tensor of magnitudes)."""
    f = torch.finfo(t)
    return torch.clamp(value.abs() * (f.eps / 2), min=f.smallest_normal * f.eps / 2)


def within(got, want, tol, what):
    got, want = got.double(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    off = ((got - want).abs() - tol)[fine]
    assert off.numel() == 0 or float(off.max()) <= 0.0, (what, float(off.max()), int((off > 0).sum()), off.numel())


def rand(shape, t, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(t)


# ---------------------------------------------------------------------------------------------------
# Norm
# ---------------------------------------------------------------------------------------------------
# every layout of a row over threads: warps, blocks, many vectors per thread, too wide for registers,
# scalar (odd widths)
WIDTHS = [1, 2, 7, 8, 31, 64, 100, 128, 129, 200, 256, 513, 640, 1000, 1024, 1283, 2048, 2051, 4096, 5000, 8191, 8192,
          8200, 16384, 16392, 32768, 33000, 40001]
TYPES = [(BF, BF), (HF, HF), (SP, SP), (BF, SP), (HF, SP)]


def norm_ref(h, w, offset, eps):
    h = h.double()
    rstd = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
    ww = (w.double() if w is not None else torch.ones((), dtype=torch.float64, device=h.device)) + offset
    return h * rstd * ww, rstd.squeeze(-1)


def check_forward(x, w, r, *, eps=1e-6, offset=0.0):
    got = F.flce_add_rms_norm(x, w, r, eps=eps, weight_offset=offset)
    if r is not None:
        assert got.h.dtype == r.dtype and torch.equal(got.h, (x.float() + r.float()).to(r.dtype))
    else:
        assert got.h is x
    y, rstd = norm_ref(got.h, w, offset, eps)
    within(got.rstd, rstd.reshape(-1), rstd.reshape(-1).abs() * 2.0 ** -17, "rstd")
    within(got.y, y, half_step(x.dtype, y) + y.abs() * 2.0 ** -17, "y")
    assert got.y.dtype == x.dtype and got.y.shape == x.shape
    return got


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("types", TYPES, ids=lambda t: f"{t[0]}-{t[1]}".replace("torch.", ""))
def test_norm_forward(types, cols):
    t, rt = types
    rows = 13 if cols < 4096 else 3
    x, r = rand((rows, cols), t, cols), rand((rows, cols), rt, cols + 1, 3.0)
    w = rand((cols,), t if cols % 2 else SP, cols + 2)
    check_forward(x, w, r, offset=float(cols % 2))
    if t == rt:
        check_forward(x, None, None)
        check_forward(x, w, None, eps=1e-3)


def test_norm_forward_shapes_strides_and_edges():
    # one row, no rows, leading dimensions, one-dimensional
    check_forward(rand((1, 4096), BF, 1), rand((4096,), BF, 2), rand((1, 4096), BF, 3))
    check_forward(rand((2, 3, 128), BF, 1), rand((128,), BF, 2), rand((2, 3, 128), SP, 3))
    check_forward(rand((640,), HF, 1), rand((640,), HF, 2), rand((640,), HF, 3))
    e = F.flce_add_rms_norm(rand((0, 64), BF, 1), rand((64,), BF, 2), rand((0, 64), BF, 3))
    assert e.y.shape == (0, 64) and e.h.shape == (0, 64) and e.rstd.shape == (0,)
    # slices of wider matrices: aligned and misaligned rows, other strides for x and the residual
    wide, res = rand((37, 3000), BF, 4), rand((37, 2100), BF, 5)
    w = rand((2051,), BF, 6)
    check_forward(wide[:, 8:8 + 1024], w[:1024], res[:, 16:16 + 1024])
    check_forward(wide[:, 3:3 + 1024], w[1:1025], res[:, 5:5 + 1024])
    check_forward(wide[:, 3:3 + 2051], w, res[:, 1:2052])
    # one row broadcast over all
    check_forward(wide[:1, :1024].expand(9, 1024), w[:1024], res[:9, :1024])
    # zero rows, and values whose squares are large and small
    z = rand((4, 512), SP, 7)
    z[1] = 0
    z[2] *= 1e15
    z[3] *= 1e-15
    check_forward(z, rand((512,), SP, 8), None)
    with pytest.raises(ValueError, match="adjacent"):
        F.flce_add_rms_norm(rand((8, 8), BF, 1).t())
    with pytest.raises(ValueError, match="shape"):
        F.flce_add_rms_norm(rand((8, 8), BF, 1), None, rand((1, 8), BF, 1))
    with pytest.raises(ValueError, match="weight"):
        F.flce_add_rms_norm(rand((8, 8), BF, 1), rand((7,), BF, 1))
    with pytest.raises(TypeError, match="dtype"):
        F.flce_add_rms_norm(rand((8, 8), torch.float64, 1))


def test_norm_nonfinite_rows_stay_in_their_rows():
    x = rand((64, 640), BF, 1)
    x[5, 17] = float("nan")
    x[9, 3] = float("inf")
    got = F.flce_add_rms_norm(x, None, rand((64, 640), BF, 2))
    bad = ~torch.isfinite(got.y.float()).all(1)
    assert torch.isnan(got.y[5].float()).all() and torch.isnan(got.y[9, 3].float())
    assert bad.nonzero().flatten().tolist() == [5, 9]


def test_norm_row_offsets_past_32_bits():
    step = (1 << 31) + 1024
    big = torch.empty(step + 4096, dtype=BF, device="cuda")
    x = big.as_strided((2, 2048), (step, 1))
    x.copy_(rand((2, 2048), BF, 3))
    got = check_forward(x, rand((2048,), BF, 4), rand((2, 2048), BF, 5))
    F.flce_add_rms_norm_backward(x, got.h, got.rstd, rand((2048,), BF, 4))
    torch.cuda.synchronize()


@pytest.mark.parametrize("group", [0, 16, 32, 48, 64, 128])
@pytest.mark.parametrize("cols", [8, 60, 128, 640, 1000, 1283, 2048, 8192, 33000])
@pytest.mark.parametrize("types", [(BF, BF), (HF, SP), (SP, SP)], ids=["bf16", "f16-f32", "f32"])
def test_norm_fp8(types, cols, group):
    """q * scale is within half a step of e4m3 (2^-4 of the value, 2^-10 of the scale below its normal range)
    of y, and the scale is the group's largest |y| / 448."""
    t, rt = types
    rows = 11 if cols < 8192 else 3
    x, r, w = rand((rows, cols), t, 1), rand((rows, cols), rt, 2), rand((cols,), t, 3)
    x[1], r[1] = 0, 0  # an empty row: scale 0
    got = F.flce_add_rms_norm_fp8(x, w, r, group=group)
    assert torch.equal(got.h, (x.float() + r.float()).to(rt))
    y, _ = norm_ref(got.h, w, 0.0, 1e-6)
    size = group or cols
    groups = -(-cols // size)
    assert got.q.dtype == torch.float8_e4m3fn and got.q.shape == x.shape and got.scale.shape == (rows, groups)
    pad = torch.nn.functional.pad(y, (0, groups * size - cols)).view(rows, groups, size)
    scale = pad.abs().amax(2) / 448.0
    within(got.scale, scale, scale * 2.0 ** -16, "scale")
    s = got.scale.double().repeat_interleave(size, 1)[:, :cols]
    value = got.q.float().double() * s
    within(value, y, y.abs() * (2.0 ** -4 + 2.0 ** -16) + s * 2.0 ** -10, "q")
    assert torch.all(got.q[1].float() == 0) and torch.all(got.scale[1] == 0)
    # the group's largest value takes the type's largest
    top = torch.nn.functional.pad(got.q.float().abs(), (0, groups * size - cols)).view(rows, groups, size).amax(2)
    assert torch.all(top[scale > 0] == 448.0)


def check_backward(dy, h, w, dh, *, offset=0.0, eps=1e-6):
    _, rstd64 = norm_ref(h, w, offset, eps)
    rstd = rstd64.reshape(-1).float()
    got = F.flce_add_rms_norm_backward(dy, h, rstd, w, dh=dh, weight_offset=offset)
    d = h.shape[-1]
    hh, dd, rr = h.double().reshape(-1, d), dy.double().reshape(-1, d), rstd.double()[:, None]
    ww = (w.double() if w is not None else torch.ones(d, dtype=torch.float64, device=h.device)) + offset
    g, n = dd * ww, hh * rr
    c = (g * n).mean(1, keepdim=True)
    want = rr * (g - n * c)
    size = rr * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dh is not None:
        want = want + dh.double().reshape(-1, d)
        size = size + dh.double().reshape(-1, d).abs()
    tol = size * 2.0 ** -17
    within(got.dx.reshape(-1, d), want, half_step(dy.dtype, want) + tol, "dx")
    within(got.dresidual.reshape(-1, d), want, half_step(h.dtype, want) + tol, "dresidual")
    assert got.dx.dtype == dy.dtype and got.dresidual.dtype == h.dtype
    if w is not None:
        terms = dd * n
        dw = terms.sum(0)
        within(got.dweight, dw, half_step(w.dtype, dw) + terms.abs().sum(0) * ((hh.shape[0] + 64) * U + 2.0 ** -22),
               "dweight")
        assert got.dweight.dtype == w.dtype
    return got


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("types", TYPES, ids=lambda t: f"{t[0]}-{t[1]}".replace("torch.", ""))
def test_norm_backward(types, cols):
    t, rt = types
    rows = 29 if cols < 4096 else 5
    dy, h, dh = rand((rows, cols), t, 1), rand((rows, cols), rt, 2, 2.0), rand((rows, cols), rt, 3)
    w = rand((cols,), t if cols % 2 else SP, 4)
    check_backward(dy, h, w, dh, offset=float(cols % 2))
    check_backward(dy, h, None, None)


@pytest.mark.parametrize("rows,cols", [(1, 4096), (1, 7), (700, 640), (1501, 2048), (2500, 1283), (400, 33000),
                                       (5000, 8)])
def test_norm_backward_many_rows(rows, cols):
    dy, h = rand((rows, cols), BF, 1), rand((rows, cols), SP, 2, 2.0)
    got = check_backward(dy, h, rand((cols,), BF, 4), rand((rows, cols), SP, 3))
    again = F.flce_add_rms_norm_backward(
        dy, h, norm_ref(h, None, 0.0, 1e-6)[1].float(), rand((cols,), BF, 4), dh=rand((rows, cols), SP, 3))
    for a, b in zip(got, again):
        assert torch.equal(a, b)  # the same bits on every run


def test_norm_backward_edges():
    w = rand((640,), BF, 4)
    e = F.flce_add_rms_norm_backward(rand((0, 640), BF, 1), rand((0, 640), BF, 2), torch.empty(0, device="cuda"), w)
    assert e.dx.shape == (0, 640) and torch.all(e.dweight == 0)
    # slices, and a gradient that is one row for all
    wide, hw = rand((37, 3000), BF, 4), rand((37, 2100), BF, 5)
    check_backward(wide[:, 8:648], hw[:, 16:656], w, None)
    check_backward(wide[:, 3:643], hw[:, 5:645], w, wide[:, 1000:1640])
    check_backward(wide[:1, :640].expand(37, 640), hw[:, :640], w, None)
    # only what is asked for
    dy, h, rstd = rand((9, 640), BF, 1), rand((9, 640), SP, 2), torch.ones(9, device="cuda")
    g = F.flce_add_rms_norm_backward(dy, h, rstd, w, need_dx=False)
    assert g.dx is None and g.dresidual.dtype == SP and g.dweight is not None
    g = F.flce_add_rms_norm_backward(dy, h, rstd, w, need_dx=False, need_dresidual=False)
    assert g.dx is None and g.dresidual is None and g.dweight is not None
    g2 = F.flce_add_rms_norm_backward(dy, h, rstd, w, need_dweight=False)
    assert g2.dweight is None and g2.dx is not None
    with pytest.raises(ValueError, match="rstd"):
        F.flce_add_rms_norm_backward(dy, h, rstd[:8], w)
    with pytest.raises(ValueError, match="shape"):
        F.flce_add_rms_norm_backward(dy, h[:8], rstd, w)


@pytest.mark.parametrize("residual", [True, False])
def test_norm_autograd_against_differences(residual):
    """The directional derivative of a scalar of (y, h) by the kernels' gradients against central differences of
    the formula in 64 bits: the difference's truncation is of the order of the step squared (1e-8), the kernels'
    fp32 error below 1e-5 of the terms."""
    n, d = 6, 96
    x, r, w = rand((n, d), SP, 1), rand((n, d), SP, 2), rand((d,), SP, 3)
    uy, uh = rand((n, d), SP, 4), rand((n, d), SP, 5)
    leaves = [t.clone().requires_grad_(True) for t in ((x, w, r) if residual else (x, w))]
    if residual:
        y, h = F.add_rms_norm(leaves[0], leaves[1], leaves[2], weight_offset=1.0)
        loss = (y * uy).sum() + (h * uh).sum()
    else:
        loss = (F.add_rms_norm(leaves[0], leaves[1], weight_offset=1.0) * uy).sum()
    loss.backward()

    def value(x, w, r=None):
        h = x + r if r is not None else x
        y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * (w + 1.0)
        return float((y * uy.double()).sum() + ((h * uh.double()).sum() if r is not None else 0.0))

    for k in range(4):
        dirs = [rand(t.shape, SP, 10 * k + i).double() for i, t in enumerate(leaves)]
        at = [t.detach().double() for t in leaves]
        s = 1e-4
        diff = (value(*[a + s * v for a, v in zip(at, dirs)]) - value(*[a - s * v for a, v in zip(at, dirs)])) / (2 * s)
        grad = sum(float((t.grad.double() * v).sum()) for t, v in zip(leaves, dirs))
        size = sum(float((t.grad.double() * v).abs().sum()) for t, v in zip(leaves, dirs))
        assert abs(grad - diff) <= 1e-5 * size


def test_norm_autograd_matches_direct_calls():
    x, r, w = rand((50, 640), BF, 1), rand((50, 640), SP, 2), rand((640,), BF, 3)
    lx, lr, lw = (t.clone().requires_grad_(True) for t in (x, r, w))
    y, h = F.add_rms_norm(lx, lw, lr)
    dy, dh = rand((50, 640), BF, 4), rand((50, 640), SP, 5)
    torch.autograd.backward([y, h], [dy, dh])
    f = F.flce_add_rms_norm(x, w, r)
    g = F.flce_add_rms_norm_backward(dy, f.h, f.rstd, w, dh=dh)
    assert torch.equal(y, f.y) and torch.equal(h, f.h)
    assert torch.equal(lx.grad, g.dx) and torch.equal(lr.grad, g.dresidual) and torch.equal(lw.grad, g.dweight)
    # only one of the outputs used; an expanded upstream gradient; a frozen weight
    lx2, lr2 = x.clone().requires_grad_(True), r.clone().requires_grad_(True)
    y2, h2 = F.add_rms_norm(lx2, w, lr2)
    h2.sum().backward()
    assert torch.all(lx2.grad == 1) and torch.all(lr2.grad == 1)
    lx3 = x.clone().requires_grad_(True)
    y3, _ = F.add_rms_norm(lx3, w, r)
    y3.sum().backward()
    g3 = F.flce_add_rms_norm_backward(torch.ones_like(x), f.h, f.rstd, w)
    assert torch.equal(lx3.grad, g3.dx)


# ---------------------------------------------------------------------------------------------------
# Gradient norm and clipping
# ---------------------------------------------------------------------------------------------------
def check_clip(grads, max_norm, outputs=None):
    before = [g.clone() for g in grads]
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(float(F.grad_norm(grads)) - want) <= want * 2.0 ** -20
    norm = F.clip_grad_norm_(grads, max_norm, outputs=outputs)
    assert norm.shape == () and norm.dtype == SP
    assert abs(float(norm) - want) <= want * 2.0 ** -20
    c = min(1.0, max_norm / (want + 1e-6)) if max_norm < math.inf else 1.0
    for b, g, o in zip(before, grads, outputs if outputs is not None else grads):
        y = b.double() * c
        within(o, y, half_step(g.dtype, y) + y.abs() * 2.0 ** -20, "clipped")
        if outputs is not None:
            assert torch.equal(b, g)
    return norm


SHAPES = [(1,), (7,), (8,), (1000, 3), (129,), (8192,), (8193,), (16384 + 5,), (0,), (300, 257), (), (2, 2, 2)]


@pytest.mark.parametrize("count", [1, 5, 32, 33, 200, 1000])
@pytest.mark.parametrize("max_norm", [1.0, 1e9, 0.0, math.inf])
def test_clip_mixed_tensors(count, max_norm):
    types = [BF, SP, HF]
    grads = [rand(SHAPES[i % len(SHAPES)], types[i % 3], i, 10.0 ** -(i % 4)) for i in range(count)]
    check_clip(grads, max_norm)


@pytest.mark.parametrize("t", [BF, HF, SP])
def test_clip_into_a_flat_buffer(t):
    """Outputs at every alignment, between guard elements that stay as they were."""
    sizes = [1, 5000, 17, 8192, 8191, 33, 30001]
    grads = [rand((n,), t, i) for i, n in enumerate(sizes)]
    flat = torch.full((sum(sizes) + 3 * len(sizes),), 7.0, dtype=t, device="cuda")
    outs, at = [], 0
    for n in sizes:
        at += 3
        outs.append(flat[at:at + n])
        at += n
    check_clip(grads, 0.5, outs)
    at = 0
    for n in sizes:
        assert torch.all(flat[at:at + 3] == 7.0)
        at += 3 + n
    # and gradients at every alignment, in place
    check_clip([flat[i * 1000 + i: i * 1000 + i + 900] for i in range(9)], 0.5)


def test_clip_extreme_values():
    """Squares that overflow or underflow fp32, alone and beside ordinary values; empty and zero tensors."""
    for scale in (1e30, 1e-30, 3e-39):
        check_clip([rand((5000,), SP, 1) * scale], 1e-3)
    check_clip([rand((5000,), SP, 1) * 1e-30, rand((100,), SP, 2) * 1e-28], math.inf)
    check_clip([rand((5000,), BF, 1) * 1e25, rand((100,), SP, 2)], 1.0)
    z = torch.zeros(4000, device="cuda")
    assert float(check_clip([z, torch.zeros(0, device="cuda")], 1.0)) == 0.0
    assert float(F.clip_grad_norm_([torch.empty(0, device="cuda")], 1.0)) == 0.0
    assert float(F.grad_norm([torch.empty(0, device="cuda")])) == 0.0
    # a NaN spreads to every gradient, as the factor is NaN; an infinity leaves zeros beside itself
    a, b = rand((4096,), BF, 1), rand((50,), SP, 2)
    a[3] = float("nan")
    assert math.isnan(float(F.clip_grad_norm_([a, b], 1.0)))
    assert torch.isnan(a.float()).all() and torch.isnan(b).all()
    a, b = rand((4096,), BF, 1), rand((50,), SP, 2)
    a[3] = float("-inf")
    assert float(F.clip_grad_norm_([a, b], 1.0)) == math.inf
    assert torch.all(b == 0) and torch.isnan(a[3]) and torch.all(a[4:] == 0)


def test_clip_layouts_and_refusals():
    g = rand((64, 48), SP, 1)
    check_clip([g.t(), rand((4, 5, 6), BF, 2).permute(2, 0, 1)], 0.1)
    with pytest.raises(ValueError, match="dense"):
        F.grad_norm([g[:, :40]])
    with pytest.raises(ValueError, match="twice"):
        F.clip_grad_norm_([g, g], 1.0)
    with pytest.raises(ValueError, match="output"):
        F.clip_grad_norm_([g], 1.0, outputs=[g.t()])
    with pytest.raises(ValueError, match="output"):
        F.clip_grad_norm_([g], 1.0, outputs=[g.to(BF)])
    with pytest.raises(ValueError, match="outputs for"):
        F.clip_grad_norm_([g], 1.0, outputs=[])
    with pytest.raises(TypeError, match="dtype"):
        F.grad_norm([g.double()])


def test_clip_is_deterministic_and_large():
    """A tensor past 2^31 elements, and the same bits on every run."""
    n = (1 << 31) + 12345
    g = torch.full((n,), 0.5, dtype=BF, device="cuda")
    g[-1] = 1024.0
    want = math.sqrt((n - 1) * 0.25 + 1024.0 ** 2)
    a = F.grad_norm([g])
    assert abs(float(a) - want) <= want * 2.0 ** -20 and torch.equal(a, F.grad_norm([g]))
    F.clip_grad_norm_([g], want / 2)
    assert float(g[0]) == 0.25 and float(g[-1]) == 512.0 and float(g[-2]) == 0.25
    grads = [rand((100003,), SP, i) for i in range(40)]
    a, b = F.grad_norm(grads), F.grad_norm(grads)
    assert torch.equal(a, b)


# ---------------------------------------------------------------------------------------------------
# Logits
# ---------------------------------------------------------------------------------------------------
def logits_ref(z, tokens, lens, prompt, rep, pres, freq, bias_ids, bias, mask, out_t):
    """(values in 64 bits, largest magnitude on the way) by the definition, on the CPU."""
    z = z.double().cpu().clone()
    b, v = z.shape
    size = torch.where(torch.isfinite(z), z.abs(), torch.zeros_like(z))
    for i in range(b):
        if tokens is not None:
            h = tokens.shape[1]
            n = h if lens is None else min(max(int(lens[i]), 0), h)
            p = 0 if prompt is None else min(max(int(prompt[i]), 0), h)
            row = tokens[i].cpu().tolist()[:n]
            for t in set(x for x in row if 0 <= x < v):
                if rep is not None:
                    r = float(rep[i])
                    z[i, t] = z[i, t] / r if z[i, t] > 0 else z[i, t] * r
                size[i, t] = max(float(size[i, t]), abs(float(z[i, t])) if math.isfinite(z[i, t]) else 0.0)
                c = row[p:].count(t)
                if c:
                    z[i, t] -= (float(freq[i]) * c if freq is not None else 0.0)
                    z[i, t] -= float(pres[i]) if pres is not None else 0.0
                    size[i, t] += (abs(float(freq[i]) * c) if freq is not None else 0.0) + \
                        (abs(float(pres[i])) if pres is not None else 0.0)
        if bias is not None:
            for t, x in zip(bias_ids[i].tolist(), bias[i].tolist()):
                if 0 <= t < v:
                    z[i, t] += x
                    size[i, t] += abs(x)
        if mask is not None:
            words = mask[i].cpu().tolist()
            for t in range(v):
                if not (words[t // 32] >> (t % 32)) & 1:
                    z[i, t] = -math.inf
    return z, size


def check_logits(z, *, out_dtype=None, n_bias=0, **kw):
    got = F.process_logits(z, out_dtype=out_dtype, **kw)
    t = out_dtype or z.dtype
    want, size = logits_ref(z, kw.get("tokens"), kw.get("lens"), kw.get("prompt_lens"), kw.get("repetition"),
                            kw.get("presence"), kw.get("frequency"), kw.get("bias_ids"), kw.get("bias"),
                            kw.get("mask"), t)
    out = got.logits.double().cpu()
    k = 8 + (kw["bias"].shape[1] if kw.get("bias") is not None else 0)
    # from half a step beyond the type's largest value on, a value rounds to infinity
    want = torch.where(torch.isinf(want.to(t)), torch.sign(want) * math.inf, want)
    within(out, want, half_step(t, want) + size * k * U, "logits")
    assert got.logits.dtype == t
    # the greedy token and the sum are those of the values as stored
    for i in range(z.shape[0]):
        row = out[i]
        if torch.isnan(row).any():
            assert int(got.token[i]) == int(torch.isnan(row).nonzero()[0])
            assert math.isnan(float(got.lse[i]))
        elif float(row.max()) == -math.inf:
            assert int(got.token[i]) == -1 and float(got.lse[i]) == -math.inf
        else:
            assert int(got.token[i]) == int((row == row.max()).nonzero()[0])
            lse = float(torch.logsumexp(row, 0))
            assert float(got.lse[i]) == lse or abs(float(got.lse[i]) - lse) <= 2.0 ** -16 + abs(lse) * 2.0 ** -22
    return got


def options(b, v, h, k, seed, ids=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    kw = dict(tokens=(v * u(b, h).double().pow(2)).long().clamp(max=v - 1).to(ids),
              lens=(u(b) * (h + 1)).long().clamp(max=h), prompt_lens=(u(b) * h).long(), repetition=0.7 + u(b),
              presence=u(b) - 0.5, frequency=u(b) - 0.5)
    if k:
        kw["bias_ids"] = torch.randint(-2, v + 2, (b, k), generator=g, device="cuda").to(ids)
        kw["bias"] = torch.randn(b, k, generator=g, device="cuda") * 4
    kw["mask"] = torch.randint(-2 ** 31, 2 ** 31, (b, (v + 31) // 32), generator=g, device="cuda").to(torch.int32)
    return kw


@pytest.mark.parametrize("types", [(SP, None), (BF, None), (HF, None), (BF, SP), (HF, SP)],
                         ids=["f32", "bf16", "f16", "bf16-f32", "f16-f32"])
@pytest.mark.parametrize("b,v,h,k", [(1, 1, 1, 1), (3, 5, 4, 2), (2, 31, 9, 0), (2, 32, 9, 3), (4, 1000, 50, 40),
                                     (3, 1023, 300, 5), (2, 1024, 300, 33), (1, 5000, 2000, 300), (5, 2049, 64, 64)])
def test_logits(types, b, v, h, k):
    t, o = types
    kw = options(b, v, h, k, v + b, torch.int64 if v % 2 else torch.int32)
    check_logits(rand((b, v), t, v, 3.0), out_dtype=o, **kw)
    kw.pop("mask")
    check_logits(rand((b, v), t, v + 1, 3.0), out_dtype=o, **kw)


@pytest.mark.parametrize("b,v", [(2, 40000), (700, 1100), (40, 20011)])
def test_logits_many_tiles_and_rows(b, v):
    """Several tiles per row, and batches whose rows are cut into few; only the options' cheap ones, so that the
    definition on the CPU stays quick."""
    z = rand((b, v), BF, v, 3.0)
    kw = options(b, v, 20, 4, v)
    kw.pop("mask")
    check_logits(z, **kw)
    check_logits(z)


def test_logits_single_options():
    """Each option alone; a history without penalties changes nothing."""
    b, v = 3, 700
    z = rand((b, v), SP, 1, 3.0)
    full = options(b, v, 60, 10, 2)
    hist = {k: full[k] for k in ("tokens", "lens", "prompt_lens")}
    assert torch.equal(check_logits(z, **hist).logits, z)
    assert torch.equal(check_logits(z, tokens=full["tokens"]).logits, z)
    for name in ("repetition", "presence", "frequency"):
        check_logits(z, **hist, **{name: full[name]})
        check_logits(z, tokens=full["tokens"], **{name: full[name]})
    check_logits(z, bias_ids=full["bias_ids"], bias=full["bias"])
    check_logits(z, mask=full["mask"])
    empty = torch.empty(b, 0, dtype=torch.int64, device="cuda")
    assert torch.equal(check_logits(z, tokens=empty, repetition=full["repetition"]).logits, z)
    assert torch.equal(check_logits(z, bias_ids=empty, bias=torch.empty(b, 0, device="cuda")).logits, z)
    r = F.process_logits(z[:0])
    assert r.logits.shape == (0, v) and r.token.shape == (0,) and r.lse.shape == (0,)


def test_logits_history_lengths_and_padding():
    """Lengths of zero, one, all and beyond; a prompt longer than the history; negative lengths; padding ids."""
    b, v, h = 7, 300, 40
    z = rand((b, v), SP, 1, 3.0)
    kw = options(b, v, h, 0, 2)
    kw.pop("mask")
    kw["lens"] = torch.tensor([0, 1, h, h + 9, -3, 20, 20], device="cuda")
    kw["prompt_lens"] = torch.tensor([0, 0, h, 5, 2, 30, -1], device="cuda")
    kw["tokens"][5, ::3] = -100
    kw["tokens"][6, ::2] = v
    kw["tokens"][2, 7] = torch.iinfo(torch.int64).min
    kw["tokens"][2, 8] = torch.iinfo(torch.int64).max
    check_logits(z, **kw)
    # one id again and again
    kw["tokens"][:] = 17
    check_logits(z, **kw)


@pytest.mark.parametrize("t", [SP, HF])
@pytest.mark.parametrize("v", [1021, 2046, 2047, 2048, 4093, 8185, 8190, 8191, 8192])
def test_logits_padding_beyond_a_vocabulary_that_ends_near_a_tile(t, v):
    """Ids at and far beyond the vocabulary are padding also where the last tile has few entries or none, for
    histories of one round and of several."""
    for h in (40, 1500):
        kw = options(2, v, h, 6, v)
        pad = torch.tensor([v, v + 1, v + 7, v + 8192, 2 ** 31 - 1, -1, 2 ** 40], device="cuda")
        kw["tokens"][:, 3:3 + len(pad)] = pad
        kw["bias_ids"][:, :2] = pad[2:4]
        kw["lens"][:] = h
        check_logits(rand((2, v), t, v, 3.0), **kw)


def test_logits_long_histories():
    """Histories of several rounds per block, crowded at a few ids, on one tile to many."""
    for b, v, h, ids in ((1, 700, 5000, torch.int64), (3, 9000, 9001, torch.int32), (2, 70001, 3000, torch.int64),
                         (40, 4100, 1025, torch.int32)):
        kw = options(b, v, h, 3, v, ids)
        kw["tokens"][:, ::3] = 1
        kw["lens"][0] = h
        kw.pop("mask")
        check_logits(rand((b, v), BF, v, 3.0), **kw)


def test_logits_duplicate_biases_add_in_order():
    z = torch.zeros(1, 64, device="cuda")
    ids = torch.tensor([[5] * 40 + [6, 5, 6]], device="cuda")
    b = rand((1, 43), SP, 1, 100.0)
    got = F.process_logits(z, bias_ids=ids, bias=b).logits[0]
    for t in (5, 6):
        s = torch.zeros((), dtype=SP)
        for i, x in zip(ids[0].tolist(), b[0].cpu()):
            if i == t:
                s = s + x
        assert float(got[t]) == float(s)


@pytest.mark.parametrize("t", [SP, BF, HF])
def test_logits_masks_infinities_and_nan(t):
    b, v = 9, 1500
    z = rand((b, v), t, 1, 3.0)
    mask = torch.full((b, (v + 31) // 32), -1, dtype=torch.int32, device="cuda")
    mask[0] = 0                                    # nothing allowed
    mask[1] = 0
    mask[1, 20] = 1 << 7                           # one entry
    z[2] = -math.inf                               # nothing finite
    z[3, 5] = math.inf
    z[4, 900] = math.nan
    z[5, 100:110], z[5, 200:210] = math.nan, math.inf
    mask[5, 100 // 32:110 // 32 + 1] = 0           # NaN and infinities in masked places only
    mask[5, 200 // 32:210 // 32 + 1] = 0
    z[6] = torch.finfo(t).min                      # the type's lowest everywhere
    z[7] = torch.finfo(t).min
    z[7, 1499] = 0.0
    z[8, 3] = z[8, 77] = z[8, 1400] = 30.0         # ties
    got = check_logits(z, mask=mask)
    assert got.token.tolist()[:2] == [-1, 20 * 32 + 7] and int(got.token[2]) == -1
    assert got.token.tolist()[3:5] == [5, 900] and int(got.token[8]) == 3
    assert int(got.token[6]) == 0 and int(got.token[7]) == 1499
    kw = options(b, v, 30, 8, 5)
    kw["mask"] = mask
    z[4, 900] = 0
    check_logits(z, **kw)


def test_logits_strides_and_in_place():
    b, v = 6, 1000
    kw = options(b, v, 30, 8, 5)
    wide = rand((b, 1300), BF, 1, 3.0)
    want = F.process_logits(wide[:, 8:8 + v].contiguous(), **kw)
    for at in (8, 1, 3):
        z = torch.empty(b, 1300, dtype=BF, device="cuda")
        z[:, at:at + v] = wide[:, 8:8 + v]
        got = F.process_logits(z[:, at:at + v], **kw)
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        # into a wider buffer, whose other columns stay
        buf = torch.full((b, 1290), 5.0, dtype=BF, device="cuda")
        F.process_logits(z[:, at:at + v], out=buf[:, 2 * at:2 * at + v], **kw)
        assert torch.equal(buf[:, 2 * at:2 * at + v], want.logits)
        assert torch.all(buf[:, :2 * at] == 5.0) and torch.all(buf[:, 2 * at + v:] == 5.0)
        # in place
        F.process_logits(z[:, at:at + v], out=z[:, at:at + v], **kw)
        assert torch.equal(z[:, at:at + v], want.logits)
    # strided options, and one row of logits for all requests
    hist = torch.full((b, 100), 3, dtype=torch.int64, device="cuda")
    hist[:, 40:70] = kw["tokens"]
    m = torch.full((b, 50), -1, dtype=torch.int32, device="cuda")
    m[:, 10:42] = kw["mask"]
    kw2 = dict(kw, tokens=hist[:, 40:70], mask=m[:, 10:42])
    for x, y in zip(F.process_logits(wide[:, 8:8 + v], **kw2), want):
        assert torch.equal(x, y)
    one = wide[:1, :v].expand(b, v)
    for x, y in zip(F.process_logits(one, **kw), F.process_logits(one.contiguous(), **kw)):
        assert torch.equal(x, y)


def test_logits_offsets_past_32_bits():
    step, v = (1 << 31) + 1000, 4096
    big = torch.empty(step + v, dtype=BF, device="cuda")
    z = big.as_strided((2, v), (step, 1))
    z.copy_(rand((2, v), BF, 3, 3.0))
    kw = options(2, v, 50, 4, 6)
    a, b = F.process_logits(z, **kw), F.process_logits(z.contiguous(), **kw)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_logits_refusals():
    z = rand((2, 64), BF, 1)
    kw = options(2, 64, 8, 3, 1)
    bad = [dict(repetition=kw["repetition"]), dict(tokens=kw["tokens"], lens=kw["lens"].int()),
           dict(tokens=kw["tokens"].float()), dict(tokens=kw["tokens"][:1]), dict(bias=kw["bias"]),
           dict(bias_ids=kw["bias_ids"], bias=kw["bias"][:, :2]), dict(mask=kw["mask"][:, :1]),
           dict(mask=kw["mask"].long()), dict(out=torch.empty(2, 63, dtype=BF, device="cuda")),
           dict(out=torch.empty(64, 2, dtype=BF, device="cuda").t()),
           dict(tokens=kw["tokens"], repetition=kw["repetition"].half())]
    for b in bad:
        with pytest.raises(ValueError, match="flce"):
            F.process_logits(z, **b)
    with pytest.raises(RuntimeError, match="do not match"):
        F.process_logits(z, out_dtype=HF)
    with pytest.raises(RuntimeError, match="CUDA"):
        F.process_logits(z, tokens=kw["tokens"].cpu())
    with pytest.raises(ValueError, match="workspace"):
        F.process_logits(z, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------------------------------------------
# Streams, graphs, memory
# ---------------------------------------------------------------------------------------------------
def _all_calls():
    x, r, w = rand((40, 640), BF, 1), rand((40, 640), BF, 2), rand((640,), BF, 3)
    rstd = torch.ones(40, device="cuda")
    grads = [rand((5000,), BF, 4), rand((77, 13), SP, 5)]
    outs = [torch.empty_like(g) for g in grads]
    z, kw = rand((3, 2000), SP, 6), options(3, 2000, 50, 7, 7)

    def calls():
        a = F.flce_add_rms_norm(x, w, r)
        q = F.flce_add_rms_norm_fp8(x, w, r)
        g = F.flce_add_rms_norm_backward(x, r, rstd, w, dh=r)
        n = F.clip_grad_norm_(grads, 0.5, outputs=outs)
        p = F.process_logits(z, **kw)
        return [a.y, a.h, a.rstd, q.q.view(torch.uint8), q.scale, g.dx, g.dweight, n, *outs, p.logits, p.token, p.lse]
    return calls


def test_other_streams_and_graph_replay_give_the_same_bits():
    calls = _all_calls()
    want = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [t.clone() for t in calls()]
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, held):
        assert torch.equal(a, b)


def test_host_memory_is_refused_before_any_launch(lib):
    import ctypes

    from linear_cross_entropy_tmem_gb300 import binding as B
    pinned = torch.zeros(64, 64, dtype=SP).pin_memory().data_ptr()
    dev = rand((64, 64), SP, 1)
    d = dev.data_ptr()
    p = B.FlceNormProblem(rows=64, cols=64, x_stride=64, y_stride=64, eps=1e-6)
    before = lib.flce_testing_launch_count()
    assert lib.flce_add_rms_norm(ctypes.byref(p), pinned, None, None, None, d, None, None) == B.FLCE_ERR_INVALID_ARG
    assert lib.flce_add_rms_norm(ctypes.byref(p), d, None, None, None, pinned, None, None) == B.FLCE_ERR_INVALID_ARG
    q = B.FlceLogitsProblem(rows=64, vocab=64, logits_stride=64, out_stride=64)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    for a in (dict(logits=pinned), dict(out=pinned), dict(mask=pinned), dict(token=pinned), dict(ws=pinned)):
        v = dict(logits=d, tokens=None, lens=None, prompt_lens=None, rep=None, pres=None, freq=None, bias_ids=None,
                 bias=None, mask=None, out=d, token=None, lse=None, ws=ws.data_ptr(), size=1 << 16)
        v.update(a)
        assert lib.flce_process_logits(ctypes.byref(q), *v.values(), None) == B.FLCE_ERR_INVALID_ARG
    one = (ctypes.c_int64 * 1)
    for src, dst in ((pinned, d), (d, pinned)):
        assert lib.flce_clip_grad_norm(one(src), one(dst), one(64), (ctypes.c_int32 * 1)(0), 1, 1.0, d, ws.data_ptr(),
                                       1 << 16, None) == B.FLCE_ERR_INVALID_ARG
    assert lib.flce_testing_launch_count() == before
    torch.cuda.synchronize()


@pytest.mark.parametrize("types", [(BF, BF), (HF, SP), (SP, SP)])
@pytest.mark.parametrize("rows,cols", [(500, 9001), (333, 16384), (320, 8200)])
def test_norm_backward_wide_many_rows(rows, cols, types):
    """Several wide rows per block: their dweight sums wait in shared memory."""
    t, rt = types
    dy, h, dh = rand((rows, cols), t, 1), rand((rows, cols), rt, 2, 2.0), rand((rows, cols), rt, 3)
    check_backward(dy, h, rand((cols,), t, 4), dh)
