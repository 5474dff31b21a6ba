"""Argument checks of the operators on either side of the head (CPU only: every refusal comes before any CUDA
call), and the layout of their parameter structs."""
from __future__ import annotations

import ctypes

import pytest
import torch

import linear_cross_entropy_tmem_gb300 as F
from linear_cross_entropy_tmem_gb300 import binding as B


def _a(i, off=0):
    return 0x100000 * (i + 1) + off


def _norm(**kw):
    base = dict(rows=4, cols=64, x_stride=64, residual_stride=64, h_stride=64, y_stride=64, dresidual_stride=64,
                dtype=B.FLCE_BF16, residual_dtype=B.FLCE_BF16, weight_dtype=B.FLCE_BF16, quant_group=0, eps=1e-6,
                weight_offset=0.0)
    base.update(kw)
    return B.FlceNormProblem(**base)


def _logits(**kw):
    base = dict(rows=2, vocab=100, history=8, n_bias=4, logits_stride=100, out_stride=100, tokens_stride=8,
                bias_ids_stride=4, bias_stride=4, mask_stride=4, logits_dtype=B.FLCE_F32, out_dtype=B.FLCE_F32,
                tokens_i64=1, bias_ids_i64=1)
    base.update(kw)
    return B.FlceLogitsProblem(**base)


def test_struct_layouts():
    assert ctypes.sizeof(B.FlceNormProblem) == 7 * 8 + 4 * 4 + 2 * 4
    assert ctypes.sizeof(B.FlceLogitsProblem) == 10 * 8 + 4 * 4


BAD_NORM = [
    (dict(rows=-1), B.FLCE_ERR_INVALID_ARG),
    (dict(rows=1 << 31), B.FLCE_ERR_INVALID_ARG),
    (dict(cols=0), B.FLCE_ERR_INVALID_ARG),
    (dict(cols=131073), B.FLCE_ERR_INVALID_ARG),
    (dict(x_stride=-1), B.FLCE_ERR_INVALID_ARG),
    (dict(eps=-1e-6), B.FLCE_ERR_INVALID_ARG),
    (dict(eps=float("nan")), B.FLCE_ERR_INVALID_ARG),
    (dict(weight_offset=float("inf")), B.FLCE_ERR_INVALID_ARG),
    (dict(dtype=3), B.FLCE_ERR_UNSUPPORTED_DTYPE),
    (dict(residual_dtype=-1), B.FLCE_ERR_UNSUPPORTED_DTYPE),
    (dict(residual_dtype=B.FLCE_F16), B.FLCE_ERR_DTYPE_MISMATCH),
    (dict(dtype=B.FLCE_F32), B.FLCE_ERR_DTYPE_MISMATCH),
]


@pytest.mark.parametrize("kw,code", BAD_NORM)
def test_norm_problem_refusals(lib, kw, code):
    p = ctypes.byref(_norm(**kw))
    n = ctypes.c_size_t()
    assert lib.flce_add_rms_norm_workspace_size(p, ctypes.byref(n)) == code
    assert lib.flce_add_rms_norm(p, _a(0), _a(1), _a(2), _a(3), _a(4), None, None) == code
    assert lib.flce_add_rms_norm_fp8(p, _a(0), _a(1), _a(2), _a(3), _a(4), _a(5), None) == code
    assert lib.flce_add_rms_norm_backward(p, _a(0), _a(1), _a(2), _a(3), None, _a(4), None, _a(5), _a(6), 1 << 30,
                                          None) == code


def test_norm_call_refusals(lib):
    p = ctypes.byref(_norm())
    fwd = lib.flce_add_rms_norm
    inv, mis = B.FLCE_ERR_INVALID_ARG, B.FLCE_ERR_MISALIGNED
    assert fwd(None, _a(0), None, None, None, _a(4), None, None) == inv
    assert fwd(p, None, _a(1), _a(2), _a(3), _a(4), None, None) == inv          # no x
    assert fwd(p, _a(0), _a(1), _a(2), _a(3), None, None, None) == inv          # no y
    assert fwd(p, _a(0), _a(1), _a(2), None, _a(4), None, None) == inv          # a residual without h
    assert fwd(p, _a(0), None, _a(2), _a(3), _a(4), None, None) == inv          # h without a residual
    assert fwd(p, _a(0, 1), _a(1), _a(2), _a(3), _a(4), None, None) == mis
    assert fwd(p, _a(0), _a(1), _a(2, 1), _a(3), _a(4), None, None) == mis
    assert fwd(p, _a(0), _a(1), _a(2), _a(3), _a(4), _a(5, 2), None) == mis
    assert fwd(ctypes.byref(_norm(y_stride=63)), _a(0), _a(1), _a(2), _a(3), _a(4), None, None) == inv
    assert fwd(ctypes.byref(_norm(h_stride=0)), _a(0), _a(1), _a(2), _a(3), _a(4), None, None) == inv
    assert fwd(ctypes.byref(_norm(weight_dtype=7)), _a(0), _a(1), _a(2), _a(3), _a(4), None, None) \
        == B.FLCE_ERR_UNSUPPORTED_DTYPE
    f32r = ctypes.byref(_norm(residual_dtype=B.FLCE_F32))
    assert fwd(f32r, _a(0), None, _a(2), None, _a(4), None, None) == B.FLCE_ERR_DTYPE_MISMATCH
    assert fwd(f32r, _a(0), _a(1, 2), _a(2), _a(3), _a(4), None, None) == mis
    assert fwd(ctypes.byref(_norm(rows=0)), None, None, None, None, None, None, None) == B.FLCE_OK
    fp8 = lib.flce_add_rms_norm_fp8
    assert fp8(p, _a(0), _a(1), _a(2), _a(3), _a(4), None, None) == inv         # no scale
    for g in (-16, 8, 100):
        assert fp8(ctypes.byref(_norm(quant_group=g)), _a(0), _a(1), _a(2), _a(3), _a(4), _a(5), None) == inv
    bwd = lib.flce_add_rms_norm_backward
    n = ctypes.c_size_t()
    assert lib.flce_add_rms_norm_workspace_size(p, ctypes.byref(n)) == B.FLCE_OK and n.value >= 4 * 64 * 4
    assert lib.flce_add_rms_norm_workspace_size(p, None) == inv
    assert bwd(p, None, _a(1), _a(2), _a(3), None, _a(4), None, _a(5), _a(6), n.value, None) == inv
    assert bwd(p, _a(0), _a(1), _a(2), None, None, _a(4), None, _a(5), _a(6), n.value, None) == inv
    assert bwd(p, _a(0), _a(1), _a(2), _a(3), None, None, None, None, _a(6), n.value, None) == inv  # nothing asked for
    assert bwd(p, _a(0), _a(1), _a(2), _a(3), None, _a(4), None, _a(5), None, n.value, None) == inv
    assert bwd(p, _a(0), _a(1), _a(2), _a(3), None, _a(4), None, _a(5), _a(6), n.value - 1, None) \
        == B.FLCE_ERR_WORKSPACE_TOO_SMALL
    assert bwd(p, _a(0), _a(1), _a(2), _a(3), _a(7, 1), _a(4), None, _a(5), _a(6), n.value, None) == mis
    assert bwd(ctypes.byref(_norm(dresidual_stride=10)), _a(0), _a(1), _a(2), _a(3), None, _a(4), _a(7), _a(5), _a(6),
               n.value, None) == inv


def _grads(n=2, numel=8, dtype=B.FLCE_F32, src=None, dst=None):
    p = ctypes.c_int64 * n
    return (p(*(src or [_a(i) for i in range(n)])), p(*(dst or [_a(i + 10) for i in range(n)])),
            p(*([numel] * n)), (ctypes.c_int32 * n)(*([dtype] * n)))


def test_clip_refusals(lib):
    inv = B.FLCE_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    assert lib.flce_grad_norm_workspace_size(-1, ctypes.byref(n)) == inv
    assert lib.flce_grad_norm_workspace_size(3, None) == inv
    assert lib.flce_grad_norm_workspace_size(2, ctypes.byref(n)) == B.FLCE_OK
    ws = n.value
    # partial sums: at least one for each tensor
    assert lib.flce_grad_norm_workspace_size(100000, ctypes.byref(n)) == B.FLCE_OK and n.value >= 100000 * 8

    def clip(g, max_norm=1.0, norm=_a(30), w=_a(31), size=ws, count=2):
        return lib.flce_clip_grad_norm(g[0], g[1], g[2], g[3], count, max_norm, norm, w, size, None)

    g = _grads()
    assert clip(g, max_norm=-1.0) == inv and clip(g, max_norm=float("nan")) == inv
    assert clip(g, norm=None) == inv and clip(g, w=None) == inv and clip(g, count=-1) == inv
    assert clip(g, size=ws - 1) == B.FLCE_ERR_WORKSPACE_TOO_SMALL
    assert clip(_grads(dtype=5)) == B.FLCE_ERR_UNSUPPORTED_DTYPE
    assert clip(_grads(numel=-1)) == inv
    assert clip(_grads(numel=1 << 62)) == inv
    assert clip(_grads(numel=(1 << 30) * 8192 - 1)) == inv  # more chunks together than the kernels count
    assert clip(_grads(src=[_a(0), 0])) == inv and clip(_grads(dst=[0, _a(1)])) == inv
    assert clip(_grads(src=[_a(0), _a(1, 2)])) == B.FLCE_ERR_MISALIGNED
    assert clip(_grads(dst=[_a(0), _a(1, 1)])) == B.FLCE_ERR_MISALIGNED
    assert lib.flce_clip_grad_norm(g[0], None, g[2], g[3], 2, 1.0, _a(30), _a(31), ws, None) == inv
    assert lib.flce_grad_norm(None, g[2], g[3], 2, _a(30), _a(31), ws, None) == inv
    assert lib.flce_grad_norm(g[0], g[2], g[3], 2, _a(30, 2), _a(31), ws, None) == B.FLCE_ERR_MISALIGNED


BAD_LOGITS = [
    (dict(rows=-1), B.FLCE_ERR_INVALID_ARG),
    (dict(rows=1 << 40), B.FLCE_ERR_INVALID_ARG),
    (dict(vocab=0), B.FLCE_ERR_INVALID_ARG),
    (dict(vocab=(1 << 30) + 1), B.FLCE_ERR_INVALID_ARG),
    (dict(history=-1), B.FLCE_ERR_INVALID_ARG),
    (dict(n_bias=-1), B.FLCE_ERR_INVALID_ARG),
    (dict(logits_stride=-100), B.FLCE_ERR_INVALID_ARG),
    (dict(out_stride=99), B.FLCE_ERR_INVALID_ARG),
    (dict(mask_stride=-4), B.FLCE_ERR_INVALID_ARG),
    (dict(logits_dtype=3), B.FLCE_ERR_UNSUPPORTED_DTYPE),
    (dict(out_dtype=-1), B.FLCE_ERR_UNSUPPORTED_DTYPE),
    (dict(out_dtype=B.FLCE_BF16), B.FLCE_ERR_DTYPE_MISMATCH),
    (dict(logits_dtype=B.FLCE_BF16, out_dtype=B.FLCE_F16), B.FLCE_ERR_DTYPE_MISMATCH),
]


def _call(lib, p, **kw):
    a = dict(logits=_a(0), tokens=_a(1), lens=_a(2), prompt_lens=_a(3), repetition=_a(4), presence=_a(5),
             frequency=_a(6), bias_ids=_a(7), bias=_a(8), mask=_a(9), out=_a(10), token=_a(11), lse=_a(12),
             ws=_a(13), size=1 << 40)
    a.update(kw)
    return lib.flce_process_logits(ctypes.byref(p), *a.values(), None)


@pytest.mark.parametrize("kw,code", BAD_LOGITS)
def test_logits_problem_refusals(lib, kw, code):
    p = _logits(**kw)
    n = ctypes.c_size_t()
    assert lib.flce_process_logits_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code
    assert _call(lib, p) == code


def test_logits_call_refusals(lib):
    p = _logits()
    inv = B.FLCE_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    assert lib.flce_process_logits_workspace_size(ctypes.byref(p), ctypes.byref(n)) == B.FLCE_OK
    assert lib.flce_process_logits_workspace_size(ctypes.byref(p), None) == inv
    for name in ("logits", "out", "ws", "bias", "bias_ids"):
        assert _call(lib, p, **{name: None}) == inv, name
    assert _call(lib, p, tokens=None) == inv  # penalties without a history
    assert _call(lib, p, size=n.value - 1) == B.FLCE_ERR_WORKSPACE_TOO_SMALL
    for name, off in (("logits", 2), ("tokens", 4), ("lens", 4), ("repetition", 1), ("bias_ids", 4), ("bias", 2),
                      ("mask", 2), ("out", 2), ("token", 4), ("lse", 2), ("ws", 8)):
        assert _call(lib, p, **{name: _a(20, off)}) == B.FLCE_ERR_MISALIGNED, name
    assert _call(lib, _logits(rows=0), logits=None, out=None, ws=None) == B.FLCE_OK


def test_python_calls_refuse_cpu_tensors():
    x = torch.zeros(2, 8)
    for call in (lambda: F.add_rms_norm(x), lambda: F.flce_add_rms_norm(x), lambda: F.flce_add_rms_norm_fp8(x),
                 lambda: F.flce_add_rms_norm_backward(x, x, torch.zeros(2)), lambda: F.grad_norm([x]),
                 lambda: F.clip_grad_norm_([x], 1.0), lambda: F.process_logits(x)):
        with pytest.raises(RuntimeError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="no gradients"):
        F.grad_norm([])
    with pytest.raises(ValueError, match="max_norm"):
        F.clip_grad_norm_([x], -1.0)
