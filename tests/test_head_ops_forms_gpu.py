"""The kernels of the norm, the clipping and the logits in the forms that larger calls take: several rows per block or
warp, tiles of every size, buffers that are read and written in place.  Formulas in 64 bits on the GPU.

Tolerances are those of test_head_ops_gpu.py.  A code of the 8-bit norm is bounded more closely: with
q = (h_j w_j) / max_j |h_j w_j| * 448 the row's rstd cancels, and what is left are the roundings of two products on
either side (4 u, and 1 u where an offset is added to the weights), of the scale (1 u) and of the corrected quotient
(1 u), u = 2^-24: at most 8 u.  So a code other than the definition's may only appear where the quotient lies within
2^-20 of itself from a border between two codes.

The norm of gradients is within 2^-20: the squares round (1 u), a thread adds 32 of them in eight chains and a tree (6 u),
its rounds compensated (2 u), and the block in two trees (10 u), fp64 from there on: at most 19 u of the sum, of which
the root keeps half.
"""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import linear_cross_entropy_tmem_gb300 as F
from linear_cross_entropy_tmem_gb300 import binding as B
from linear_cross_entropy_tmem_gb300 import head_ops

from .test_head_ops_gpu import (BF, HF, SP, U, check_backward, check_clip, check_forward, half_step, norm_ref, options,
                                rand, within)

pytestmark = pytest.mark.gpu

CODES = {SP: B.FLCE_F32, BF: B.FLCE_BF16, HF: B.FLCE_F16}
TYPES = [(BF, BF), (HF, SP), (SP, SP)]
IDS = ["bf16", "f16-f32", "f32"]

# Six rows or more for each warp or block of a GPU of 152 SMs: a warp per row (with whole and ragged rows), blocks of up
# to 256, 512 and 1024 threads, rows too wide for registers.
ROWS = [(40000, 128), (40000, 129), (20000, 500), (20000, 640), (16001, 1283), (6001, 2048), (6001, 2051), (6001, 4096),
        (6001, 4099), (2500, 8192), (2500, 8191), (1000, 12001), (1000, 16384), (300, 16400)]


def placed(rows, cols, t, seed, scale, at):
    """Rows within a wider matrix, `at` elements past its rows' start (None: a matrix of their own)."""
    if at is None:
        return rand((rows, cols), t, seed, scale)
    return rand((rows, (cols + at + 23) // 16 * 16), t, seed, scale)[:, at:at + cols]


# where x and the residual start: rows of their own; both shifted alike; shifted differently (single elements)
PLACES = [(None, None), (3, 3), (1, 4)]


@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("places", PLACES, ids=["own", "shifted", "single"])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_norm_forward_several_rows(types, places, rows, cols):
    t, rt = types
    x, r = placed(rows, cols, t, 1, 1.0, places[0]), placed(rows, cols, rt, 2, 3.0, places[1])
    check_forward(x, rand((cols,), t, 3), r, offset=1.0)
    if t == rt and places[0] is None:
        check_forward(x, None, None)


def codes(q):
    return torch.clamp(q, -448.0, 448.0).float().to(torch.float8_e4m3fn).float()


def check_fp8(x, w, r, group, offset=0.0):
    got = F.flce_add_rms_norm_fp8(x, w, r, group=group, weight_offset=offset)
    rows, cols = x.shape
    h = x
    if r is not None:
        h = got.h
        assert torch.equal(h, (x.float() + r.float()).to(r.dtype))
    y, _ = norm_ref(h, w, offset, 1e-6)
    size = group or cols
    groups = -(-cols // size)
    top = torch.nn.functional.pad(y, (0, groups * size - cols)).view(rows, groups, size).abs().amax(2)
    within(got.scale, top / 448.0, top / 448.0 * 2.0 ** -16, "scale")
    q = torch.where(y == 0, torch.zeros_like(y), y / (top / 448.0).repeat_interleave(size, 1)[:, :cols])
    a, b, g = codes(q * (1 - 2.0 ** -20)), codes(q * (1 + 2.0 ** -20)), got.q.float()
    bad = (g != a) & (g != b)
    assert not bad.any(), (int(bad.sum()), g[bad][:4], q[bad][:4])
    return got


@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("group", [0, 16, 48, 128])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_norm_fp8_several_rows(types, group, rows, cols):
    t, rt = types
    # columns and rows of very different size, so that a maximum of the row before shows
    scale = torch.exp(2.0 * rand((rows, 1), SP, 5))
    x, r = rand((rows, cols), t, 1), (rand((rows, cols), SP, 2) * scale).to(rt)
    x[7::11], r[7::11] = 0, 0
    got = check_fp8(x, rand((cols,), t, 3), r, group, offset=float(cols % 2))
    assert torch.all(got.scale[7::11] == 0) and torch.all(got.q[7::11].float() == 0)


@pytest.mark.parametrize("group", [0, 48, 128])
@pytest.mark.parametrize("places", PLACES[1:], ids=["shifted", "single"])
@pytest.mark.parametrize("rows,cols", [(20000, 500), (16001, 1283), (6001, 2048), (2500, 8191)])
def test_norm_fp8_several_rows_placed(rows, cols, places, group):
    check_fp8(placed(rows, cols, BF, 1, 1.0, places[0]), rand((cols,), BF, 3), placed(rows, cols, BF, 2, 3.0, places[1]),
              group)


@pytest.mark.parametrize("rows,cols,group", [(8192, 2048, 128), (8192, 2048, 0), (4096, 4096, 32), (40000, 128, 64),
                                             (16001, 1283, 48), (2500, 8191, 128), (1000, 16384, 128), (300, 33000, 16),
                                             (3, 131072, 16)])
@pytest.mark.parametrize("types", [(BF, BF, BF), (HF, HF, HF), (BF, BF, SP), (HF, SP, HF), (SP, SP, SP)],
                         ids=["bf16", "f16", "bf16-weights-f32", "f16-f32", "f32"])
def test_norm_fp8_codes_are_the_quotients(types, rows, cols, group):
    """Every code is that of the quotient in 64 bits rounded to fp32.  The kernel's quotient is within 2^-44 of itself
    before its one rounding to fp32; to give another code it would have to round to the other side of one of e4m3's
    borders, for which the chance is below 2^-40 an element, 2^-15 a test."""
    t, rt, wt = types
    x, r, w = rand((rows, cols), t, 1), rand((rows, cols), rt, 2, 2.0), rand((cols,), wt, 3)
    for offset in (0.0, 1.0):
        if offset:  # multiples of 2^-6: exact when 1 is added
            w = ((w.float() * 64.0).round() / 64.0).to(wt)
        got = F.flce_add_rms_norm_fp8(x, w, r, group=group, weight_offset=offset)
        y, size = norm_ref(got.h, w, offset, 1e-6)[0], group or cols
        groups = -(-cols // size)
        top = torch.nn.functional.pad(y, (0, groups * size - cols)).view(rows, groups, size).abs().amax(2)
        want = codes(y / (top / 448.0).repeat_interleave(size, 1)[:, :cols])
        assert int((got.q.float() != want).sum()) == 0


@pytest.mark.parametrize("t,wt", [(BF, BF), (BF, SP), (SP, SP)], ids=["bf16", "bf16-weights-f32", "f32"])
@pytest.mark.parametrize("size", [1e-35, 1e-25, 1e15])
@pytest.mark.parametrize("cols,group", [(2048, 128), (2048, 0), (1283, 48), (16400, 64)])
def test_norm_fp8_codes_of_small_and_large_rows(t, wt, size, cols, group):
    """The same for values whose reciprocals, squares or products come near fp32's ends."""
    x, w = (rand((40, cols), SP, 1) * size).to(t), rand((cols,), wt, 3)
    got = F.flce_add_rms_norm_fp8(x, w, None, group=group)
    y, n = norm_ref(x, w, 0.0, 1e-6)[0], group or cols
    groups = -(-cols // n)
    top = torch.nn.functional.pad(y, (0, groups * n - cols)).view(40, groups, n).abs().amax(2)
    want = codes(y / (top / 448.0).repeat_interleave(n, 1)[:, :cols])
    assert int((got.q.float() != want).sum()) == 0
    within(got.scale, top / 448.0, top / 448.0 * 2.0 ** -16, "scale")


@pytest.mark.parametrize("t,rt", [(BF, BF), (HF, SP)], ids=["bf16", "f16-f32"])
@pytest.mark.parametrize("cols,group", [(2048, 128), (2048, 48), (1283, 128), (16400, 128)])
def test_norm_fp8_groups_without_a_finite_maximum(t, rt, cols, group):
    x, r, w = rand((5, cols), t, 1), rand((5, cols), rt, 2), rand((cols,), t, 3)
    clean = F.flce_add_rms_norm_fp8(x, w, r, group=group)
    x[1, 200] = math.nan           # the whole row
    x[2, 300] = math.inf           # rstd 0: the infinity's group is NaN, the others are 0
    w2 = w.clone()
    w2[70] = math.inf              # that group of every row
    got = F.flce_add_rms_norm_fp8(x, w, r, group=group)
    assert torch.isnan(got.scale[1]).all() and torch.isnan(got.q[1].float()).all()
    at = 300 // group
    rest = [g for g in range(got.scale.shape[1]) if g != at]
    assert torch.isnan(got.scale[2, at]) and torch.all(got.scale[2, rest] == 0)
    q = got.q[2].float()
    assert torch.isnan(q[300]) and torch.all(torch.cat([q[:at * group], q[(at + 1) * group:]]) == 0)
    for row in (0, 3, 4):
        assert torch.equal(got.q[row].view(torch.uint8), clean.q[row].view(torch.uint8))
        assert torch.equal(got.scale[row], clean.scale[row])
    got = F.flce_add_rms_norm_fp8(x, w2, r, group=group)
    at = 70 // group
    assert not torch.isfinite(got.scale[:, at]).any() and torch.isnan(got.q[0, 70].float())
    keep = [g for g in range(got.scale.shape[1]) if g != at]
    assert torch.equal(got.scale[0, keep], clean.scale[0, keep])


@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("places", PLACES, ids=["own", "shifted", "single"])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_norm_backward_several_rows(types, places, rows, cols):
    t, rt = types
    check_backward(placed(rows, cols, t, 1, 1.0, places[0]), placed(rows, cols, rt, 2, 2.0, places[1]),
                   rand((cols,), t, 3), placed(rows, cols, rt, 4, 1.0, places[1]), offset=1.0)


# ---------------------------------------------------------------------------------------------------
# In place
# ---------------------------------------------------------------------------------------------------
def norm_problem(rows, cols, t, rt, strides, wt=None):
    return B.FlceNormProblem(rows=rows, cols=cols, x_stride=strides[0], residual_stride=strides[1], h_stride=strides[2],
                             y_stride=strides[3], dresidual_stride=strides[4], dtype=CODES[t], residual_dtype=CODES[rt],
                             weight_dtype=CODES[wt or t], eps=1e-6)


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("rows,cols", ROWS + [(5, 33000), (3, 640)])
@pytest.mark.parametrize("at", [None, 3])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_norm_forward_in_place(lib, types, at, rows, cols):
    """y in x's memory and h in the residual's: the bits of a call with buffers of their own, nothing beside them."""
    t, rt = types
    x, r, w = placed(rows, cols, t, 1, 1.0, at), placed(rows, cols, rt, 2, 3.0, at), rand((cols,), t, 3)
    want = F.flce_add_rms_norm(x, w, r)
    # out of place into matrices of their own the vectors may be laid out otherwise: the same layout first
    y, h = torch.empty_strided(x.shape, x.stride(), dtype=t, device="cuda"), torch.empty_strided(
        r.shape, r.stride(), dtype=rt, device="cuda")
    rstd, rstd2 = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    p = ctypes.byref(norm_problem(rows, cols, t, rt, (x.stride(0), r.stride(0), r.stride(0), x.stride(0), 0)))
    around = [(b, b.clone()) for b in (x._base, r._base) if b is not None]
    assert lib.flce_add_rms_norm(p, x.data_ptr(), r.data_ptr(), w.data_ptr(), h.data_ptr(), y.data_ptr(),
                                 rstd.data_ptr(), stream()) == B.FLCE_OK
    assert lib.flce_add_rms_norm(p, x.data_ptr(), r.data_ptr(), w.data_ptr(), r.data_ptr(), x.data_ptr(),
                                 rstd2.data_ptr(), stream()) == B.FLCE_OK
    assert torch.equal(r, want.h) and torch.equal(h, r)
    ref, rstd64 = norm_ref(r, w, 0.0, 1e-6)
    for got in (x, y):
        within(got, ref, half_step(t, ref) + ref.abs() * 2.0 ** -17, "y")
    within(rstd2, rstd64, rstd64 * 2.0 ** -17, "rstd")
    if at is None:  # alike in layout as well
        assert torch.equal(x, y) and torch.equal(x, want.y) and torch.equal(rstd, rstd2)
    for now, before in around:
        assert torch.equal(now[:, :at], before[:, :at]) and torch.equal(now[:, at + cols:], before[:, at + cols:])


@pytest.mark.parametrize("rows,cols", ROWS + [(5, 33000), (3, 640)])
@pytest.mark.parametrize("at", [None, 3])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
def test_norm_backward_in_place(lib, types, at, rows, cols):
    """dx in dy's memory and dresidual in dh's, with dweight: the bits of a call with buffers of their own."""
    t, rt = types
    dy, h, dh = placed(rows, cols, t, 1, 1.0, at), placed(rows, cols, rt, 2, 2.0, at), placed(rows, cols, rt, 4, 1.0, at)
    w = rand((cols,), t, 3)
    rstd = norm_ref(h, w, 0.0, 1e-6)[1].float()
    p = ctypes.byref(norm_problem(rows, cols, t, rt,
                                  (dy.stride(0), dh.stride(0), h.stride(0), dy.stride(0), dh.stride(0))))
    size = ctypes.c_size_t()
    assert lib.flce_add_rms_norm_workspace_size(p, ctypes.byref(size)) == B.FLCE_OK
    ws = torch.empty(size.value, dtype=torch.uint8, device="cuda")
    # the same alignment as in place
    own = lambda a: torch.empty_like(a._base)[:, at:at + cols] if at else torch.empty_like(a)  # noqa: E731
    dx, dr, dw, dw2 = own(dy), own(dh), torch.empty_like(w), torch.empty_like(w)
    around = [(b, b.clone()) for b in (dy._base, dh._base) if b is not None]

    def call(x, r, dw):
        assert lib.flce_add_rms_norm_backward(p, dy.data_ptr(), h.data_ptr(), w.data_ptr(), rstd.data_ptr(),
                                              dh.data_ptr(), x.data_ptr(), r.data_ptr(), dw.data_ptr(), ws.data_ptr(),
                                              size.value, stream()) == B.FLCE_OK
    call(dx, dr, dw)
    call(dy, dh, dw2)
    assert torch.equal(dy, dx) and torch.equal(dh, dr) and torch.equal(dw, dw2)
    for now, before in around:
        assert torch.equal(now[:, :at], before[:, :at]) and torch.equal(now[:, at + cols:], before[:, at + cols:])


def test_norm_backward_row_offsets_past_32_bits():
    step, cols = (1 << 31) + 1024, 2048
    big = torch.empty(step + 4 * cols, dtype=BF, device="cuda")
    dy, h, dh = (big[k * cols:].as_strided((2, cols), (step, 1)) for k in range(3))
    for k, a in enumerate((dy, h, dh)):
        a.copy_(rand((2, cols), BF, k + 1))
    check_backward(dy, h, rand((cols,), BF, 4), dh)


# ---------------------------------------------------------------------------------------------------
# Clipping
# ---------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("t,small", [(SP, 1e-16), (SP, 1e-30), (BF, 1e-16), (BF, 1e-30)])
def test_clip_sizes_mixed_within_a_tensor(t, small):
    """Stretches whose squares vanish in fp32 beside ordinary ones, within a chunk and as whole chunks."""
    g = rand((300, 1000), SP, 1, 1e-2)
    g[10:20] *= small
    g[100:250] *= small
    g[::7, ::3] *= small
    check_clip([g.to(t), rand((77,), t, 2)], 0.5)
    check_clip([g.to(t)[100:250].clone(), g.to(t)[10:11].clone()], 0.5 * small)


def test_clip_norm_beyond_fp32():
    """A norm above fp32's largest value is infinite, though no gradient is: the factor is 0."""
    a, b = torch.full((2,), 3e38, device="cuda"), rand((50,), BF, 1)
    assert float(F.grad_norm([a, b])) == math.inf
    assert float(F.clip_grad_norm_([a, b], 1.0)) == math.inf
    assert torch.all(a == 0) and torch.all(b == 0)


# ---------------------------------------------------------------------------------------------------
# Logits
# ---------------------------------------------------------------------------------------------------
def logits_reference(z, kw):
    """(values in 64 bits, largest magnitude on the way) by the definition, for all rows at once."""
    z = z.double()
    b, v = z.shape
    size = z.abs()

    def spread(ids, x):  # sums of x by id; ids outside the vocabulary are padding
        inside = (ids >= 0) & (ids < v)
        return torch.zeros(b, v, dtype=torch.float64, device="cuda").scatter_add_(
            1, torch.where(inside, ids, torch.zeros_like(ids)).long(), torch.where(inside, x.double(), 0.0))
    t = kw["tokens"]
    at = torch.arange(t.shape[1], device="cuda")[None]
    live = at < kw["lens"].clamp(0, t.shape[1])[:, None]
    seen = spread(t, live) > 0
    n = spread(t, live & (at >= kw["prompt_lens"].clamp(0, t.shape[1])[:, None]))
    r, f, p = (kw[k].double()[:, None] for k in ("repetition", "frequency", "presence"))
    z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
    size = torch.maximum(size, z.abs())
    z = z - f * n - torch.where(n > 0, p, 0.0)
    size = size + (f * n).abs() + torch.where(n > 0, p.abs(), 0.0)
    if kw.get("bias") is not None:
        z = z + spread(kw["bias_ids"], kw["bias"])
        size = size + spread(kw["bias_ids"], kw["bias"].abs())
    if kw.get("mask") is not None:
        bits = (kw["mask"].long()[:, :, None] >> torch.arange(32, device="cuda")) & 1
        z = torch.where(bits.view(b, -1)[:, :v] > 0, z, -math.inf)
    return z, size


def check_rows(got, z, kw):
    want, size = logits_reference(z, kw)
    out = got.logits.double()
    k = 8 + (kw["bias"].shape[1] if kw.get("bias") is not None else 0)
    within(out, want, half_step(got.logits.dtype, want) + size * k * U, "logits")
    top = out.amax(1)
    first = torch.where(out == top[:, None], torch.arange(z.shape[1], device="cuda")[None], z.shape[1]).amin(1)
    assert torch.equal(got.token, torch.where(top == -math.inf, -1, first))
    lse = torch.logsumexp(out, 1)
    within(got.lse, lse, 2.0 ** -16 + lse.abs() * 2.0 ** -22, "lse")
    return first


# 32, 16, 8 and 4 entries per thread of 256 (three blocks for each of 152 SMs or more), on one tile to several
SIZES = [(500, 8200), (500, 20011), (500, 8192), (200, 10001), (200, 10240), (100, 10001), (100, 10240), (40, 5003)]


@pytest.mark.parametrize("b,v", SIZES)
@pytest.mark.parametrize("single", [False, True], ids=["vectors", "single"])
@pytest.mark.parametrize("types", [(SP, SP), (BF, BF), (HF, HF), (BF, SP), (HF, SP)],
                         ids=["f32", "bf16", "f16", "bf16-f32", "f16-f32"])
def test_logits_tiles(types, single, b, v):
    """Histories, repeated and padding biases, masks, and equal maxima in other vectors and tiles."""
    t, o = types
    for h, k, mask in ((300, 6, True), (2600, 0, True), (40, 600, False)):
        kw = options(b, v, h, k, v + h, torch.int64 if h > 300 else torch.int32)
        kw["tokens"][:, ::5] = v + kw["tokens"][:, ::5] % 40  # padding
        kw["tokens"][:, 1::6] = kw["tokens"][:, :1] % 50      # crowded
        kw["lens"][::3] = h
        kw["lens"][1::5] = 0
        if k:
            kw["bias_ids"][:, 1] = kw["bias_ids"][:, 0]       # twice
            kw["bias_ids"][1::10] = -1                        # none
        if not mask:
            kw.pop("mask")
        else:
            kw["mask"][2::9] = 0
        z = rand((b, v), t, v, 3.0)
        g = torch.Generator(device="cuda").manual_seed(h)
        ties = torch.randint(0, v, (b, 40), generator=g, device="cuda")
        z.scatter_(1, ties, 60.0)
        if mask:
            kw["mask"].scatter_(1, ties // 32, -1)
            kw["mask"][4::9] = 0                              # nothing allowed
        out = None
        if single:  # a row of out begins elsewhere in its 16 bytes than the logits' row
            out = torch.full((b, (v + 24) // 8 * 8), 7.0, dtype=o, device="cuda")
            out = out[:, 1:1 + v] if v % 8 == 0 else out[:, 3:3 + v]
        got = F.process_logits(z, out=out, out_dtype=o, **kw)
        check_rows(got, z, kw)
        if single:
            assert torch.all(out._base[:, :1] == 7.0) and torch.all(out._base[:, -4:] == 7.0)
        elif t == o:  # in place, with the same layout
            again = F.process_logits(z, out=z, **kw)
            assert torch.equal(z.view(torch.uint8), got.logits.view(torch.uint8))
            assert torch.equal(again.token, got.token) and torch.equal(again.lse, got.lse)


def test_logits_equal_maxima_of_rows_without_options():
    """Every pair of places in a row of several tiles: the lower one."""
    b, v = 500, 20011
    for t in (SP, BF):
        z = rand((b, v), t, 1)
        i = torch.arange(b, device="cuda")
        lo, hi = (i * 37) % 9000, 9001 + (i * 83) % 11000
        z[i, lo], z[i, hi] = 40.0, 40.0
        assert torch.equal(F.process_logits(z).token, lo)


# ---------------------------------------------------------------------------------------------------
# Native and Python marshalling
# ---------------------------------------------------------------------------------------------------
def test_both_ways_of_marshalling_agree(monkeypatch):
    x, r, w = rand((5, 7, 130), BF, 1), rand((5, 7, 130), SP, 2), rand((130,), HF, 3)
    dy, dh = rand((5, 7, 130), BF, 4), rand((5, 7, 130), SP, 5)
    z, kw = rand((4, 999), HF, 6), options(4, 999, 30, 5, 7)
    grads = [rand(s, t, 8) for s, t in (((50, 3), BF), ((), SP), ((0,), HF), ((9000,), HF))]

    def run():
        f = F.flce_add_rms_norm(x, w, r, weight_offset=1.0, eps=1e-5)
        f0 = F.flce_add_rms_norm(x, None, None, need_rstd=False)
        assert f0.h is x and f0.rstd is None
        q = [F.flce_add_rms_norm_fp8(x, w, r, group=g) for g in (0, 32)]
        b = F.flce_add_rms_norm_backward(dy, f.h, f.rstd, w, dh=dh, weight_offset=1.0)
        b2 = F.flce_add_rms_norm_backward(dy, x, f.rstd, w, need_dresidual=False)
        assert b2.dresidual is None
        own = [g.clone() for g in grads]
        n = F.clip_grad_norm_(own, 0.25)
        out = torch.empty(4, 999, dtype=SP, device="cuda")
        p = F.process_logits(z, out=out, **kw)
        assert p.logits is out
        p2 = F.process_logits(z, out_dtype=SP, mask=kw["mask"])
        return [*f, f0.y, *q[0], *q[1], *b, b2.dx, b2.dweight, n, F.grad_norm(grads), *own, *p, *p2]
    native = run()
    monkeypatch.setattr(head_ops, "_call", lambda *a: None)
    for a, b in zip(native, run()):
        assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride()
        assert torch.equal(a.contiguous().view(torch.uint8) if a.dim() else a, b.contiguous().view(torch.uint8) if b.dim() else b)
