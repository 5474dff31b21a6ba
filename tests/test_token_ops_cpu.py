"""Argument checks of the operators that lead from one token to the next (CPU only: every refusal comes before any CUDA
call), and the layout of their parameter structs."""
from __future__ import annotations

import ctypes

import pytest
import torch

import linear_cross_entropy_tmem_gb300 as F
from linear_cross_entropy_tmem_gb300 import binding as B

INV, MIS, TYPE = B.FLCE_ERR_INVALID_ARG, B.FLCE_ERR_MISALIGNED, B.FLCE_ERR_UNSUPPORTED_DTYPE


def _a(i, off=0):
    return 0x100000 * (i + 1) + off


def _embedding(**kw):
    base = dict(tokens=4, vocab=100, cols=64, weight_stride=64, out_stride=64, padding=-1, weight_dtype=B.FLCE_BF16,
                out_dtype=B.FLCE_BF16, ids_i64=1, accumulate=0, scale=1.0)
    base.update(kw)
    return B.FlceEmbeddingProblem(**base)


def _mx(**kw):
    base = dict(rows=4, cols=64, stride=64, dtype=B.FLCE_BF16)
    base.update(kw)
    return B.FlceMxfp4Problem(**base)


def _mx_logits(**kw):
    base = dict(tokens=4, vocab=1000, cols=64, hidden_stride=64, out_stride=1000, hidden_dtype=B.FLCE_BF16,
                out_dtype=B.FLCE_F32, bias_dtype=B.FLCE_BF16, logit_scale=1.0, softcap=0.0)
    base.update(kw)
    return B.FlceMxfp4LogitsProblem(**base)


def _sample(**kw):
    base = dict(rows=4, vocab=1000, logits_stride=1000, logits_dtype=B.FLCE_F32)
    base.update(kw)
    return B.FlceSampleProblem(**base)


def test_struct_layouts():
    assert ctypes.sizeof(B.FlceEmbeddingProblem) == 6 * 8 + 4 * 4 + 4 + 4
    assert ctypes.sizeof(B.FlceMxfp4Problem) == 3 * 8 + 2 * 4
    assert ctypes.sizeof(B.FlceMxfp4LogitsProblem) == 5 * 8 + 3 * 4 + 2 * 4 + 4
    assert ctypes.sizeof(B.FlceSampleProblem) == 3 * 8 + 2 * 4


BAD_EMBEDDING = [
    (dict(tokens=-1), INV),
    (dict(tokens=(1 << 30) + 1), INV),
    (dict(vocab=0), INV),
    (dict(vocab=(1 << 31) - 1), INV),
    (dict(cols=0), INV),
    (dict(cols=(1 << 24) + 1), INV),
    (dict(weight_stride=-1), INV),
    (dict(out_stride=-64), INV),
    (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV),
    (dict(weight_dtype=3), TYPE),
    (dict(out_dtype=-1), TYPE),
    (dict(out_dtype=B.FLCE_F16), B.FLCE_ERR_DTYPE_MISMATCH),
    (dict(weight_dtype=B.FLCE_F32), B.FLCE_ERR_DTYPE_MISMATCH),
]


@pytest.mark.parametrize("kw,code", BAD_EMBEDDING)
def test_embedding_problem_refusals(lib, kw, code):
    p = ctypes.byref(_embedding(**kw))
    n = ctypes.c_size_t()
    assert lib.flce_embedding(p, _a(0), _a(1), _a(2), None) == code
    assert lib.flce_embedding_workspace_size(p, ctypes.byref(n)) == code
    assert lib.flce_embedding_backward(p, _a(0), _a(1), _a(2), _a(3), 1 << 40, None) == code


def test_embedding_call_refusals(lib):
    p = ctypes.byref(_embedding())
    fwd, bwd = lib.flce_embedding, lib.flce_embedding_backward
    assert fwd(None, _a(0), _a(1), _a(2), None) == INV
    for i in range(3):
        assert fwd(p, *(None if i == k else _a(k) for k in range(3)), None) == INV
    assert fwd(p, _a(0, 4), _a(1), _a(2), None) == MIS
    assert fwd(p, _a(0), _a(1, 1), _a(2), None) == MIS
    assert fwd(p, _a(0), _a(1), _a(2, 1), None) == MIS
    assert fwd(ctypes.byref(_embedding(out_stride=63)), _a(0), _a(1), _a(2), None) == INV
    assert fwd(ctypes.byref(_embedding(tokens=1 << 30, cols=1 << 24, out_stride=1 << 24)), _a(0), _a(1), _a(2), None) == INV
    assert fwd(ctypes.byref(_embedding(tokens=0)), None, None, None, None) == B.FLCE_OK
    n = ctypes.c_size_t()
    assert lib.flce_embedding_workspace_size(p, None) == INV
    assert lib.flce_embedding_workspace_size(p, ctypes.byref(n)) == B.FLCE_OK and n.value >= 4 * 16
    for i in range(4):
        assert bwd(p, *(None if i == k else _a(k) for k in range(4)), n.value, None) == INV
    assert bwd(p, _a(0), _a(1), _a(2), _a(3), n.value - 1, None) == B.FLCE_ERR_WORKSPACE_TOO_SMALL
    for i, off in ((0, 4), (1, 1), (2, 1), (3, 8)):
        assert bwd(p, *(_a(k, off if i == k else 0) for k in range(4)), n.value, None) == MIS
    assert bwd(ctypes.byref(_embedding(weight_stride=63)), _a(0), _a(1), _a(2), _a(3), n.value, None) == INV
    # nothing to add, nothing to do
    assert bwd(ctypes.byref(_embedding(tokens=0, accumulate=1)), None, None, None, None, n.value, None) == B.FLCE_OK
    # nothing but zeros to write, and nowhere to
    assert bwd(ctypes.byref(_embedding(tokens=0)), None, None, None, _a(3), n.value, None) == INV


BAD_MX = [
    (dict(rows=-1), INV),
    (dict(rows=(1 << 31) - 1), INV),
    (dict(cols=0), INV),
    (dict(cols=(1 << 24) + 1), INV),
    (dict(rows=1 << 30, cols=1 << 24), INV),
    (dict(stride=-1), INV),
    (dict(dtype=3), TYPE),
]


@pytest.mark.parametrize("kw,code", BAD_MX)
def test_mxfp4_refusals(lib, kw, code):
    p = ctypes.byref(_mx(**kw))
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.flce_mxfp4_quantize(p, _a(0), _a(1), _a(2), None) == code
    assert lib.flce_mxfp4_dequantize(p, _a(0), _a(1), _a(2), None) == code
    if "stride" not in kw and "dtype" not in kw:
        assert lib.flce_mxfp4_size(p, ctypes.byref(a), ctypes.byref(b)) == code


def test_mxfp4_call_refusals(lib):
    p = ctypes.byref(_mx())
    q, d = lib.flce_mxfp4_quantize, lib.flce_mxfp4_dequantize
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.flce_mxfp4_size(None, ctypes.byref(a), ctypes.byref(b)) == INV
    assert lib.flce_mxfp4_size(p, None, ctypes.byref(b)) == INV
    assert lib.flce_mxfp4_size(ctypes.byref(_mx(rows=129, cols=33)), ctypes.byref(a), ctypes.byref(b)) == B.FLCE_OK
    assert (a.value, b.value) == (129 * 32, 2 * 512)
    for call in (q, d):
        for i in range(3):
            assert call(p, *(None if i == k else _a(k) for k in range(3)), None) == INV
        assert call(ctypes.byref(_mx(rows=0)), None, None, None, None) == B.FLCE_OK
    for i, off in ((0, 1), (1, 8), (2, 8)):
        assert q(p, *(_a(k, off if i == k else 0) for k in range(3)), None) == MIS
    for i, off in ((0, 8), (1, 8), (2, 1)):
        assert d(p, *(_a(k, off if i == k else 0) for k in range(3)), None) == MIS
    assert d(ctypes.byref(_mx(stride=63)), _a(0), _a(1), _a(2), None) == INV


BAD_MX_LOGITS = [
    (dict(tokens=-1), INV),
    (dict(tokens=(1 << 24) + 1), INV),
    (dict(vocab=0), INV),
    (dict(vocab=(1 << 31) - 256), INV),
    (dict(cols=0), INV),
    (dict(cols=(1 << 20) + 1), INV),
    (dict(tokens=1 << 24, vocab=1 << 30), INV),
    (dict(hidden_stride=-1), INV),
    (dict(out_stride=-1), INV),
    (dict(logit_scale=float("nan")), INV),
    (dict(softcap=-1.0), INV),
    (dict(softcap=float("inf")), INV),
    (dict(hidden_dtype=3), TYPE),
    (dict(out_dtype=-1), TYPE),
    (dict(bias_dtype=9), TYPE),
]


@pytest.mark.parametrize("kw,code", BAD_MX_LOGITS)
def test_mxfp4_logits_problem_refusals(lib, kw, code):
    p = ctypes.byref(_mx_logits(**kw))
    n = ctypes.c_size_t()
    assert lib.flce_mxfp4_logits_workspace_size(p, ctypes.byref(n)) == code
    assert lib.flce_mxfp4_logits(p, *(_a(k) for k in range(6)), 1 << 40, None) == code


def test_mxfp4_logits_call_refusals(lib):
    p = ctypes.byref(_mx_logits())
    f = lib.flce_mxfp4_logits
    n = ctypes.c_size_t()
    assert lib.flce_mxfp4_logits_workspace_size(p, None) == INV
    assert lib.flce_mxfp4_logits_workspace_size(p, ctypes.byref(n)) == B.FLCE_OK
    for i in (0, 1, 2, 4, 5):  # (3: no bias)
        assert f(p, *(None if i == k else _a(k) for k in range(6)), n.value, None) == INV
    for i, off in ((0, 1), (1, 8), (2, 8), (3, 1), (4, 2), (5, 8)):
        assert f(p, *(_a(k, off if i == k else 0) for k in range(6)), n.value, None) == MIS
    assert f(p, *(_a(k) for k in range(6)), n.value - 1, None) == B.FLCE_ERR_WORKSPACE_TOO_SMALL
    assert f(ctypes.byref(_mx_logits(out_stride=999)), *(_a(k) for k in range(6)), n.value, None) == INV
    assert f(ctypes.byref(_mx_logits(tokens=0)), None, None, None, None, None, None, n.value, None) == B.FLCE_OK
    # the workspace holds the hidden states in 4 bits
    big = ctypes.c_size_t()
    assert lib.flce_mxfp4_logits_workspace_size(ctypes.byref(_mx_logits(tokens=2047, cols=4096)), ctypes.byref(big)) == B.FLCE_OK
    assert 2047 * 4096 * 17 // 32 <= big.value <= 2 * 2047 * 4096


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INV), (dict(rows=1 << 31), INV), (dict(vocab=0), INV), (dict(vocab=(1 << 20) + 1), INV),
    (dict(logits_stride=-1), INV), (dict(logits_dtype=3), TYPE)])
def test_sample_problem_refusals(lib, kw, code):
    assert lib.flce_sample(ctypes.byref(_sample(**kw)), *(_a(k) for k in range(9)), None) == code


def test_sample_call_refusals(lib):
    p = ctypes.byref(_sample())
    f = lib.flce_sample
    assert f(None, *(_a(k) for k in range(9)), None) == INV
    for i in (0, 1, 6):
        assert f(p, *(None if i == k else _a(k) for k in range(9)), None) == INV
    for i, off in ((0, 2), (1, 2), (2, 2), (3, 4), (4, 2), (5, 2), (6, 4), (7, 2), (8, 4)):
        assert f(p, *(_a(k, off if i == k else 0) for k in range(9)), None) == MIS
    assert f(ctypes.byref(_sample(rows=0)), *([None] * 9), None) == B.FLCE_OK


def test_python_calls_refuse_cpu_tensors():
    w, ids, u = torch.zeros(4, 64), torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    q = F.MxFp4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), 64)
    assert q.shape == (4, 64)
    for call in (lambda: F.embedding(w, ids), lambda: F.flce_embedding(w, ids),
                 lambda: F.flce_embedding_backward(w[:2], ids, 4), lambda: F.mxfp4_quantize(w),
                 lambda: F.mxfp4_dequantize(q), lambda: F.mxfp4_logits(w, q), lambda: F.sample_tokens(w[:2], u)):
        with pytest.raises(RuntimeError, match="CUDA"):
            call()
