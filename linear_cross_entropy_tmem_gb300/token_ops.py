"""Torch-facing calls of the operators that lead from one token to the next: argument checks and marshalling only.

* :func:`embedding` (autograd), :func:`flce_embedding` and :func:`flce_embedding_backward`: rows of a table by token,
  scaled, and the table's gradient (which can be added to a head's, where the table is the head's weight).
* :func:`mxfp4_quantize`, :func:`mxfp4_dequantize` and :func:`mxfp4_logits`: a head whose weight is held in 4 bits.
* :func:`sample_tokens`: temperature, top-k, top-p and min-p on logits, and the token that a given random number chooses.

As in ``head_ops.py``, PyTorch provides device memory and the current stream, every step runs in ``libflce.so``, and
there is no CPU path.  See ``include/flce.h`` for the formulas.  Tensors that are as the library wants them are
marshalled by ``flce_torch``; it returns None for the others, which the code here views as rows, or refuses.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import NamedTuple, Optional

import torch
from torch.autograd.graph import increment_version

from . import binding as B
from .head_ops import _addr, _adjacent, _call, _code, _on, _rows, _stream, _workspace
from .once import once

_IDS = (torch.int64, torch.int32)


# ---------------------------------------------------------------------------------------------------
# Embedding
# ---------------------------------------------------------------------------------------------------
@lru_cache(maxsize=256)
def _embedding_problem(*fields):
    return B.FlceEmbeddingProblem(*fields, 0)


def _flat_ids(ids):
    if ids.dtype not in _IDS:
        raise TypeError(f"flce: ids: dtype {ids.dtype} is not supported (int64 or int32)")
    if not ids.is_contiguous():
        raise ValueError("flce: ids must be contiguous")
    return ids.numel()


def _want(dtype, what):
    return -1 if dtype is None else _code(dtype, what)


def _pad(padding_idx):
    if padding_idx is None:
        return -1
    if padding_idx < 0:  # (torch's embedding counts it from the table's end; here -1 is what tokens without an id have)
        raise ValueError(f"flce: padding_idx must be None or an id of the table, got {padding_idx}: negative numbers are "
                         "not counted from its end")
    return int(padding_idx)


def flce_embedding(weight: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0,
                   out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """``weight[ids] * scale`` (see ``flce_embedding`` in include/flce.h): [..., D] for ids of any shape.  Rows of ids
    outside [0, V), such as the -1 of :func:`process_logits` and :func:`sample_tokens`, are zeros.  ``out_dtype`` is
    the weight's dtype or fp32.  The result carries no gradient: :func:`embedding` is the call for autograd."""
    res = _call("embedding", weight, ids, scale, _want(out_dtype, "out"))
    if res is not None:
        return res[0]
    dev = weight.device
    _on(dev, weight=weight, ids=ids)
    if weight.dim() != 2 or weight.shape[0] == 0 or weight.shape[1] == 0:
        raise ValueError("flce: weight must be a matrix with at least one row and one column")
    w = _rows(weight, "weight")
    n, (v, d) = _flat_ids(ids), w.shape
    out = torch.empty(*ids.shape, d, dtype=out_dtype or weight.dtype, device=dev)
    prob = _embedding_problem(n, v, d, w.stride(0), d, -1, _code(weight.dtype, "weight"), _code(out.dtype, "out"),
                              int(ids.dtype == torch.int64), 0, float(scale))
    B.check(B.load().flce_embedding(ctypes.byref(prob), _addr(ids), _addr(w), _addr(out), _stream(dev)),
            "flce_embedding")
    return out


def flce_embedding_backward(dout: torch.Tensor, ids: torch.Tensor, vocab: int, *, scale: float = 1.0,
                            padding_idx: Optional[int] = None, dtype: Optional[torch.dtype] = None,
                            dweight: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient [vocab, D] of the table, from that of the rows (see ``flce_embedding_backward``), in ``dtype`` (dout's).
    With ``dweight``, a matrix such as the gradient that a tied head's backward left, the rows' sums are added to it
    in place (rows without a token are left as they are), and it is returned.  ``padding_idx``: as in
    :func:`embedding`."""
    res = _call("embedding_backward", dout, ids, vocab, scale, _pad(padding_idx), _want(dtype, "dweight"), dweight,
                workspace)
    if res is not None:
        return res[0]
    dev = dout.device
    _on(dev, dout=dout, ids=ids, dweight=dweight)
    d2 = _rows(dout, "dout")
    n, d = d2.shape
    if d == 0:
        raise ValueError("flce: dout must have at least one column")
    if _flat_ids(ids) != n or dout.shape[:-1] != ids.shape:
        raise ValueError(f"flce: dout has shape {tuple(dout.shape)}, ids {tuple(ids.shape)}")
    vocab = int(vocab)
    given = dweight is not None
    if given:
        if dweight.shape != (vocab, d) or (dtype is not None and dweight.dtype != dtype) or \
                (d > 1 and dweight.stride(1) != 1):
            raise ValueError(f"flce: dweight must be a {dtype or ''} matrix of {vocab} rows of {d} adjacent elements")
    elif not 1 <= vocab < 2 ** 31 - 1:
        raise ValueError(f"flce: vocab must be positive and below 2^31 - 1, got {vocab}")
    else:
        dweight = torch.empty(vocab, d, dtype=dtype or dout.dtype, device=dev)
    prob = _embedding_problem(n, vocab, d, dweight.stride(0), d2.stride(0), _pad(padding_idx),
                              _code(dweight.dtype, "dweight"), _code(dout.dtype, "dout"),
                              int(ids.dtype == torch.int64), int(given), float(scale))
    lib = B.load()
    size = ctypes.c_size_t(0)
    B.check(lib.flce_embedding_workspace_size(ctypes.byref(prob), ctypes.byref(size)), "flce_embedding_workspace_size")
    ws = _workspace(size.value, dev, workspace)
    B.check(lib.flce_embedding_backward(ctypes.byref(prob), _addr(ids), _addr(d2), _addr(dweight), _addr(ws), size.value,
                                        _stream(dev)), "flce_embedding_backward")
    if given:
        increment_version(dweight)
    return dweight


class Embedding(torch.autograd.Function):
    """Autograd wrapper.  The table's gradient is dense, in its dtype; it has no derivative of its own: a second
    backward through it raises."""

    @staticmethod
    def forward(ctx, weight, ids, scale, padding_idx, out_dtype):
        _pad(padding_idx)
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.dtype, ctx.scale, ctx.padding = weight.shape[0], weight.dtype, scale, padding_idx
        return flce_embedding(weight, ids, scale=scale, out_dtype=out_dtype)

    @staticmethod
    def backward(ctx, dout):
        if not ctx.needs_input_grad[0]:
            return None, None, None, None, None
        ids, = ctx.saved_tensors
        dw = flce_embedding_backward(_adjacent(dout), ids, ctx.vocab, scale=ctx.scale, padding_idx=ctx.padding,
                                     dtype=ctx.dtype)
        return once("embedding", dw, dout), None, None, None, None


def embedding(weight: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0, padding_idx: Optional[int] = None,
              out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """``weight[ids] * scale`` with the table's gradient: rows of ids outside [0, V) are zeros, and neither they nor
    ``padding_idx`` have one (an id of the table; a negative number is refused, it does not count from the end).

    A backward captured into a CUDA graph: while an earlier graph of the same leaf lives, autograd adds to the leaf on
    the stream on which that graph was recorded.  Record it on the capturing stream, or drop it before the capture."""
    return Embedding.apply(weight, ids, float(scale), padding_idx, out_dtype)


# ---------------------------------------------------------------------------------------------------
# 4 bits
# ---------------------------------------------------------------------------------------------------
class MxFp4(NamedTuple):
    """A matrix in 4 bits with a power of two for each 32 columns of a row (layouts: ``flce_mxfp4_size``)."""
    codes: torch.Tensor   # uint8 [rows, 16 * ceil(cols / 32)]: two e2m1 codes to a byte, the even column's low
    scales: torch.Tensor  # uint8 [ceil(rows / 128), ceil(ceil(cols / 32) / 4), 32, 4, 4]: exponents + 127
    cols: int

    @property
    def shape(self):
        return self.codes.shape[0], self.cols


def _mx_layout(rows, cols):
    blocks = -(-cols // 32)
    return (rows, blocks * 16), (-(-rows // 128), -(-blocks // 4), 32, 4, 4)


def _mx_operand(q, device, name):
    _on(device, **{f"{name}.codes": q.codes, f"{name}.scales": q.scales})
    codes, scales = _mx_layout(q.codes.shape[0] if q.codes.dim() == 2 else -1, int(q.cols))
    if q.cols < 1 or q.codes.shape != codes or q.scales.shape != scales or q.codes.dtype != torch.uint8 or \
            q.scales.dtype != torch.uint8 or not q.codes.is_contiguous() or not q.scales.is_contiguous():
        raise ValueError(f"flce: {name} must hold contiguous uint8 codes [rows, {codes[1]}] and scales "
                         f"[ceil(rows / 128), {scales[1]}, 32, 4, 4] for {q.cols} columns")


def mxfp4_quantize(x: torch.Tensor) -> MxFp4:
    """``x`` [..., D] as rows in 4 bits (see ``flce_mxfp4_quantize``).  The result carries no gradient."""
    res = _call("mxfp4_quantize", x)
    if res is not None:
        return MxFp4(*res, x.shape[-1])
    dev = x.device
    _on(dev, x=x)
    x2 = _rows(x, "x")
    n, d = x2.shape
    if d == 0:
        raise ValueError("flce: x must have at least one column")
    codes, scales = _mx_layout(n, d)
    q = MxFp4(torch.empty(codes, dtype=torch.uint8, device=dev), torch.empty(scales, dtype=torch.uint8, device=dev), d)
    prob = B.FlceMxfp4Problem(n, d, x2.stride(0), _code(x.dtype, "x"), 0)
    B.check(B.load().flce_mxfp4_quantize(ctypes.byref(prob), _addr(x2), _addr(q.codes), _addr(q.scales), _stream(dev)),
            "flce_mxfp4_quantize")
    return q


def mxfp4_dequantize(q: MxFp4, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The values that ``q`` stands for, [rows, cols], rounded to ``dtype`` (fp32 and bf16 hold them exactly)."""
    res = _call("mxfp4_dequantize", q.codes, q.scales, q.cols, _code(dtype, "out"))
    if res is not None:
        return res[0]
    dev = q.codes.device
    _mx_operand(q, dev, "q")
    n, d = q.shape
    out = torch.empty(n, d, dtype=dtype, device=dev)
    prob = B.FlceMxfp4Problem(n, d, d, _code(dtype, "out"), 0)
    B.check(B.load().flce_mxfp4_dequantize(ctypes.byref(prob), _addr(q.codes), _addr(q.scales), _addr(out),
                                           _stream(dev)), "flce_mxfp4_dequantize")
    return out


@lru_cache(maxsize=256)
def _mx_logits_problem(*fields):
    return B.FlceMxfp4LogitsProblem(*fields, 0)


def mxfp4_logits(hidden: torch.Tensor, weight: MxFp4, bias: Optional[torch.Tensor] = None, *, logit_scale: float = 1.0,
                 softcap: float = 0.0, out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Logits [..., V] of hidden states [..., D] from a head's weight in 4 bits (see ``flce_mxfp4_logits``): the hidden
    states are quantised in the call, the product runs on both in 4 bits.  ``out_dtype`` is hidden's dtype, or any of
    the three; ``out`` a matrix of rows to write.  Nothing is recorded for autograd; a given ``out`` counts as changed
    in place.  The kernel's waits are bounded: to see whether it gave one up, give a ``workspace`` (of uint8) and read its
    status with :func:`flce_read_device_status`; without one the status is dropped with the call's own workspace."""
    res = _call("mxfp4_logits", hidden, weight.codes, weight.scales, weight.cols, bias, logit_scale, softcap,
                _want(out_dtype, "out"), out, workspace)
    if res is not None:
        return res[0]
    dev = hidden.device
    _on(dev, hidden=hidden, bias=bias, out=out)
    _mx_operand(weight, dev, "weight")
    h = _rows(hidden, "hidden")
    n, d = h.shape
    v = weight.codes.shape[0]
    if d != weight.cols or v == 0:
        raise ValueError(f"flce: hidden has {d} columns, the weight {weight.cols} and {v} rows")
    if bias is not None and (bias.shape != (v,) or not bias.is_contiguous()):
        raise ValueError(f"flce: bias must be a contiguous vector of {v} elements")
    given = out is not None
    if not given:
        out = torch.empty(*hidden.shape[:-1], v, dtype=out_dtype or hidden.dtype, device=dev)
        o2 = out.view(n, v) if n else out
    elif out.shape != (*hidden.shape[:-1], v) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError(f"flce: out must have shape {(*hidden.shape[:-1], v)} and out_dtype")
    else:
        o2 = _rows(out, "out")
    prob = _mx_logits_problem(n, v, d, h.stride(0), o2.stride(0) if n else v, _code(hidden.dtype, "hidden"),
                              _code(out.dtype, "out"), _code(bias.dtype, "bias") if bias is not None else B.FLCE_F32,
                              float(logit_scale), float(softcap))
    lib = B.load()
    size = ctypes.c_size_t(0)
    B.check(lib.flce_mxfp4_logits_workspace_size(ctypes.byref(prob), ctypes.byref(size)),
            "flce_mxfp4_logits_workspace_size")
    ws = _workspace(size.value, dev, workspace)
    B.check(lib.flce_mxfp4_logits(ctypes.byref(prob), _addr(h), _addr(weight.codes), _addr(weight.scales), _addr(bias),
                                  _addr(out), _addr(ws), size.value, _stream(dev)), "flce_mxfp4_logits")
    if given:
        increment_version(out)
    return out


# ---------------------------------------------------------------------------------------------------
# Sampling
# ---------------------------------------------------------------------------------------------------
class SampledTokens(NamedTuple):
    token: torch.Tensor    # [B] int64, -1 where nothing is allowed
    logprob: torch.Tensor  # [B] fp32: log-probability among the entries that stayed
    kept: torch.Tensor     # [B] int64: how many stayed


def sample_tokens(logits: torch.Tensor, uniform: torch.Tensor, *, temperature: Optional[torch.Tensor] = None,
                  top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
                  min_p: Optional[torch.Tensor] = None) -> SampledTokens:
    """A token for each row of logits [B, V], chosen by ``uniform`` [B] (fp32 in [0, 1)) among the entries that
    ``top_k`` [B] int64, then ``top_p``, then ``min_p`` [B] fp32 leave at ``temperature`` [B] fp32 (0: greedy); see
    ``flce_sample`` in include/flce.h.  Nothing is recorded for autograd."""
    res = _call("sample_tokens", logits, uniform, temperature, top_k, top_p, min_p)
    if res is not None:
        return SampledTokens._make(res)
    dev = logits.device
    _on(dev, logits=logits, uniform=uniform, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    if logits.dim() != 2 or logits.shape[1] == 0:
        raise ValueError("flce: logits must be a matrix with at least one column")
    z = _rows(logits, "logits")
    b, v = z.shape
    for name, t, dtype in (("uniform", uniform, torch.float32), ("temperature", temperature, torch.float32),
                           ("top_k", top_k, torch.int64), ("top_p", top_p, torch.float32),
                           ("min_p", min_p, torch.float32)):
        if t is not None and (t.shape != (b,) or t.dtype != dtype or not t.is_contiguous()):
            raise ValueError(f"flce: {name} must be a contiguous {dtype} vector of {b} elements")
    token = torch.empty(b, dtype=torch.int64, device=dev)
    logprob = torch.empty(b, dtype=torch.float32, device=dev)
    kept = torch.empty(b, dtype=torch.int64, device=dev)
    prob = B.FlceSampleProblem(b, v, z.stride(0), _code(logits.dtype, "logits"), 0)
    B.check(B.load().flce_sample(ctypes.byref(prob), _addr(z), _addr(uniform), _addr(temperature), _addr(top_k),
                                 _addr(top_p), _addr(min_p), _addr(token), _addr(logprob), _addr(kept), _stream(dev)),
            "flce_sample")
    return SampledTokens(token, logprob, kept)
