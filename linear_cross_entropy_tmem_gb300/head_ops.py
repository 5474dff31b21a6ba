"""Torch-facing calls of the operators on either side of the head: argument checks and marshalling only.

* :func:`add_rms_norm` (autograd), :func:`flce_add_rms_norm`, :func:`flce_add_rms_norm_backward` and
  :func:`flce_add_rms_norm_fp8`: the norm of the residual stream that makes the head's ``hidden``.
* :func:`grad_norm` and :func:`clip_grad_norm_`: the gradients that a backward left behind.
* :func:`process_logits`: penalties, biases and masks on the head's logits, the greedy token and the
  log-sum-exp.

As in ``api.py``, PyTorch provides device memory and the current stream, every step runs in
``libflce.so``, and there is no CPU path.  See ``include/flce.h`` for the formulas.

Tensors that are as the library wants them are marshalled by ``flce_torch`` (a step of one token
is shorter than reading its tensors' fields from Python); it returns None for the others, which the
code here views as rows, or refuses.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache
from typing import Iterable, NamedTuple, Optional, Sequence

import torch
from torch.autograd.graph import increment_version

from . import binding as B
from .once import once

_DTYPES = {torch.float32: B.FLCE_F32, torch.bfloat16: B.FLCE_BF16, torch.float16: B.FLCE_F16}


def _code(dt: torch.dtype, what: str) -> int:
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError(f"flce: {what}: dtype {dt} is not supported (bf16, fp16 or fp32)")
    return code


_native = None  # flce_torch, once it is loaded


def _call(name: str, *args):
    """The outputs of a native call, or None where the tensors need a closer look."""
    global _native
    if _native is None:
        _native = B.load_torch()
    out = getattr(_native, name)(*args)
    if type(out) is int:
        raise B.FlceError(out, name)
    return out


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _on(device: torch.device, **tensors) -> None:
    """Every tensor is a CUDA tensor of the one device."""
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise RuntimeError(f"flce: {name}: inputs must be CUDA tensors (the library has no CPU path)")
        if t.device != device:
            raise ValueError(f"flce: {name} is on {t.device}, expected {device}")


def _addr(t: Optional[torch.Tensor]):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _rows(t: torch.Tensor, name: str) -> torch.Tensor:
    """``t`` as a matrix of rows whose elements are adjacent, without a copy."""
    if t.dim() == 0:
        raise ValueError(f"flce: {name} must have at least one dimension")
    if t.dim() != 2:
        try:
            t = t.view(-1, t.shape[-1]) if t.numel() else t.reshape(t.numel(), t.shape[-1])
        except RuntimeError:
            raise ValueError(f"flce: {name}: its leading dimensions cannot be viewed as rows; call "
                             ".contiguous()") from None
    if t.shape[1] > 1 and t.numel() and t.stride(1) != 1:
        raise ValueError(f"flce: the elements of a row of {name} must be adjacent")
    return t


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    _on(device, workspace=workspace)
    if not workspace.is_contiguous() or workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"flce: the workspace must be contiguous and hold {nbytes} bytes")
    return workspace


# ---------------------------------------------------------------------------------------------------
# Residual addition and root-mean-square norm
# ---------------------------------------------------------------------------------------------------
class AddRmsNormResult(NamedTuple):
    y: torch.Tensor                # normalised rows, x's dtype
    h: torch.Tensor                # x + residual in the residual's dtype (x itself without a residual)
    rstd: Optional[torch.Tensor]   # [rows] fp32, for the backward


class AddRmsNormFp8Result(NamedTuple):
    q: torch.Tensor       # float8_e4m3fn, x's shape
    scale: torch.Tensor   # fp32 [..., ceil(D / group)]: y is about q * scale
    h: torch.Tensor


class AddRmsNormGrads(NamedTuple):
    dx: Optional[torch.Tensor]
    dresidual: Optional[torch.Tensor]  # the same values in h's dtype (dx itself when the dtypes are equal)
    dweight: Optional[torch.Tensor]


def _norm_operands(x, weight, residual):
    _on(x.device, x=x, weight=weight, residual=residual)
    x2 = _rows(x, "x")
    d = x2.shape[1]
    if d == 0:
        raise ValueError("flce: x must have at least one column")
    r2 = None
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError(f"flce: residual has shape {tuple(residual.shape)}, x {tuple(x.shape)}")
        r2 = _rows(residual, "residual")
    if weight is not None and (weight.shape != (d,) or not weight.is_contiguous()):
        raise ValueError(f"flce: weight must be a contiguous vector of {d} elements")
    return x2, r2


@lru_cache(maxsize=256)
def _norm_problem(rows, cols, xs, rs, hs, ys, drs, dtype, rdtype, wdtype, group, eps, offset):
    return B.FlceNormProblem(rows=rows, cols=cols, x_stride=xs, residual_stride=rs, h_stride=hs, y_stride=ys,
                             dresidual_stride=drs, dtype=dtype, residual_dtype=rdtype, weight_dtype=wdtype,
                             quant_group=group, eps=eps, weight_offset=offset)


def _norm_forward(x, weight, residual, eps, offset, *, rstd, group=None):
    x2, r2 = _norm_operands(x, weight, residual)
    n, d = x2.shape
    code = _code(x.dtype, "x")
    wcode = _code(weight.dtype, "weight") if weight is not None else code
    rcode = _code(residual.dtype, "residual") if residual is not None else code
    y = torch.empty(x.shape, dtype=x.dtype if group is None else torch.float8_e4m3fn, device=x.device)
    h = torch.empty(x.shape, dtype=residual.dtype, device=x.device) if residual is not None else x
    prob = _norm_problem(n, d, x2.stride(0), r2.stride(0) if r2 is not None else 0, d, d, 0, code, rcode, wcode,
                         group or 0, float(eps), float(offset))
    lib = B.load()
    st = _stream(x.device)
    hp = _addr(h) if residual is not None else None
    if group is None:
        extra = torch.empty(n, dtype=torch.float32, device=x.device) if rstd else None
        B.check(lib.flce_add_rms_norm(ctypes.byref(prob), _addr(x2), _addr(r2), _addr(weight), hp, _addr(y),
                                      _addr(extra), st), "flce_add_rms_norm")
    else:
        groups = -(-d // group) if group else 1
        extra = torch.empty(*x.shape[:-1], groups, dtype=torch.float32, device=x.device)
        B.check(lib.flce_add_rms_norm_fp8(ctypes.byref(prob), _addr(x2), _addr(r2), _addr(weight), hp, _addr(y),
                                          _addr(extra), st), "flce_add_rms_norm_fp8")
    return y, h, extra


def flce_add_rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                      residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6, weight_offset: float = 0.0,
                      need_rstd: bool = True) -> AddRmsNormResult:
    """Forward of the residual addition and norm over the last dimension (see ``flce_add_rms_norm`` in
    include/flce.h); ``need_rstd=False`` where no backward follows.  Its results carry no gradient:
    :func:`add_rms_norm` is the call for autograd."""
    out = _call("add_rms_norm", x, weight, residual, eps, weight_offset, bool(need_rstd), -1)
    if out is None:
        out = _norm_forward(x, weight, residual, eps, weight_offset, rstd=need_rstd)
    return AddRmsNormResult._make(out)


def flce_add_rms_norm_fp8(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                          residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6, weight_offset: float = 0.0,
                          group: int = 128) -> AddRmsNormFp8Result:
    """The forward with an e4m3 output and one fp32 scale per ``group`` columns of a row (0: per row; see
    ``flce_add_rms_norm_fp8``).  Its results carry no gradient."""
    if not 0 <= group <= 1 << 20:
        raise ValueError(f"flce: group must be 0 or a multiple of 16, got {group}")
    out = _call("add_rms_norm", x, weight, residual, eps, weight_offset, False, int(group))
    q, h, s = out if out is not None else _norm_forward(x, weight, residual, eps, weight_offset, rstd=False,
                                                        group=int(group))
    return AddRmsNormFp8Result(q, s, h)


def flce_add_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor,
                               weight: Optional[torch.Tensor] = None, *, dh: Optional[torch.Tensor] = None,
                               weight_offset: float = 0.0, need_dx: bool = True, need_dresidual: bool = True,
                               need_dweight: bool = True, workspace: Optional[torch.Tensor] = None) -> AddRmsNormGrads:
    """Backward (see ``flce_add_rms_norm_backward``): ``dy`` is the gradient of y, ``dh`` that of h from its other
    uses; ``h`` and ``rstd`` come from the forward.  ``dx`` has dy's dtype, ``dresidual`` h's."""
    out = _call("add_rms_norm_backward", dy, h, rstd, weight, dh, weight_offset, bool(need_dx), bool(need_dresidual),
                bool(need_dweight), workspace)
    if out is not None:
        return AddRmsNormGrads._make(out)
    dev = dy.device
    _on(dev, dy=dy, h=h, rstd=rstd, weight=weight, dh=dh)
    if h.shape != dy.shape or (dh is not None and (dh.shape != dy.shape or dh.dtype != h.dtype)):
        raise ValueError("flce: dy, h and dh must have one shape, and dh h's dtype")
    dy2, h2 = _rows(dy, "dy"), _rows(h, "h")
    dh2 = _rows(dh, "dh") if dh is not None else None
    n, d = dy2.shape
    if d == 0:
        raise ValueError("flce: dy must have at least one column")
    if rstd.dtype != torch.float32 or rstd.numel() != n or not rstd.is_contiguous():
        raise ValueError(f"flce: rstd must be {n} contiguous fp32 values")
    if weight is not None and (weight.shape != (d,) or not weight.is_contiguous()):
        raise ValueError(f"flce: weight must be a contiguous vector of {d} elements")
    same = dy.dtype == h.dtype
    want = need_dx or (need_dresidual and same)
    dx = torch.empty(dy.shape, dtype=dy.dtype, device=dev) if want else None
    dr = torch.empty(h.shape, dtype=h.dtype, device=dev) if need_dresidual and not same else None
    dw = torch.empty_like(weight) if weight is not None and need_dweight else None
    code = _code(dy.dtype, "dy")
    prob = _norm_problem(n, d, dy2.stride(0), dh2.stride(0) if dh2 is not None else 0, h2.stride(0), d,
                         d if dr is not None else 0, code, _code(h.dtype, "h"),
                         _code(weight.dtype, "weight") if weight is not None else code, 0, 0.0, float(weight_offset))
    if dx is None and dr is None and dw is None:
        return AddRmsNormGrads(None, None, None)
    lib = B.load()
    ws, nbytes = None, 0
    if dw is not None:
        out = ctypes.c_size_t(0)
        B.check(lib.flce_add_rms_norm_workspace_size(ctypes.byref(prob), ctypes.byref(out)),
                "flce_add_rms_norm_workspace_size")
        nbytes = out.value
        ws = _workspace(nbytes, dev, workspace)
    B.check(lib.flce_add_rms_norm_backward(ctypes.byref(prob), _addr(dy2), _addr(h2), _addr(weight), _addr(rstd),
                                           _addr(dh2), _addr(dx), _addr(dr), _addr(dw), _addr(ws), nbytes,
                                           _stream(dev)), "flce_add_rms_norm_backward")
    return AddRmsNormGrads(dx if need_dx else None, (dx if same else dr) if need_dresidual else None, dw)


class AddRmsNorm(torch.autograd.Function):
    """Autograd wrapper: ``(y, h)`` of x and an optional residual.  The gradients of x and of the residual are
    the same values; the backward forms what is asked for.  It has no derivative of its own: a second backward
    through the gradients raises."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps, weight_offset):
        need = any(ctx.needs_input_grad[:3])
        r = flce_add_rms_norm(x, weight, residual, eps=eps, weight_offset=weight_offset, need_rstd=need)
        ctx.offset = weight_offset
        ctx.dtype = x.dtype
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        if need:
            ctx.save_for_backward(r.h if residual is not None else x, weight, r.rstd)
        if residual is None:
            return r.y
        return r.y, r.h

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        nx, nw, nr = ctx.needs_input_grad[:3]
        if dy is None and dh is None:
            return None, None, None, None, None
        if dy is None:  # only h was used
            dy = torch.zeros(h.shape, dtype=ctx.dtype, device=h.device)
        g = flce_add_rms_norm_backward(_adjacent(dy), h, rstd, weight, dh=None if dh is None else _adjacent(dh),
                                       weight_offset=ctx.offset, need_dx=nx, need_dresidual=nr and ctx.has_residual,
                                       need_dweight=nw)
        # what the gradients depend on: h only where it has a gradient itself
        stream = h if nx or nr else None
        d = (dy, dh, stream, weight)
        return (once("add_rms_norm", g.dx, *d), once("add_rms_norm", g.dweight, dy, stream),
                once("add_rms_norm", g.dresidual, *d), None, None)


def _adjacent(t: torch.Tensor) -> torch.Tensor:
    """``t``, copied when its rows are not adjacent elements (an expanded or transposed gradient)."""
    return t if t.is_contiguous() else t.contiguous()


def add_rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None, *,
                 eps: float = 1e-6, weight_offset: float = 0.0):
    """Residual addition and root-mean-square norm over the last dimension, with gradients.  Returns ``(y, h)``,
    h = x + residual being the residual stream from here on, or y alone without a residual."""
    return AddRmsNorm.apply(x, weight, residual, float(eps), float(weight_offset))


# ---------------------------------------------------------------------------------------------------
# Global gradient norm and clipping
# ---------------------------------------------------------------------------------------------------
def _dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill one stretch of memory, in any order of its dimensions."""
    if t.is_contiguous():
        return True
    size = 1
    for st, sz in sorted(zip(t.stride(), t.shape)):
        if sz != 1 and st != size:
            return False
        size *= sz
    return True


def _grad_arrays(grads: Sequence[torch.Tensor], outputs: Optional[Sequence[torch.Tensor]]):
    if not grads:
        raise ValueError("flce: no gradients")
    dev = grads[0].device
    n = len(grads)
    codes = []
    for i, g in enumerate(grads):
        if not g.is_cuda:
            raise RuntimeError("flce: gradients must be CUDA tensors (the library has no CPU path)")
        if g.device != dev:
            raise ValueError(f"flce: gradient {i} is on {g.device}, expected {dev}")
        if not _dense(g):
            raise ValueError(f"flce: gradient {i} is not dense")
        codes.append(_code(g.dtype, f"gradient {i}"))
    src = [g.data_ptr() for g in grads]
    numel = [g.numel() for g in grads]
    dst = None
    if outputs is not None:
        if len(outputs) != n:
            raise ValueError(f"flce: {len(outputs)} outputs for {n} gradients")
        for i, (g, o) in enumerate(zip(grads, outputs)):
            if o.device != dev or o.dtype != g.dtype or o.shape != g.shape or \
                    (o.stride() != g.stride() and not (o.is_contiguous() and g.is_contiguous())):
                raise ValueError(f"flce: output {i} must have its gradient's device, dtype, shape and strides")
        dst = [o.data_ptr() for o in outputs]
    live = [p for p, k in zip(dst if dst is not None else src, numel) if k]
    if len(set(live)) != len(live):
        raise ValueError("flce: the same memory appears twice among the " +
                         ("outputs" if outputs is not None else "gradients"))
    ptrs = ctypes.c_int64 * n
    arr = [ptrs(*src), ptrs(*(dst if dst is not None else src)), ptrs(*numel), (ctypes.c_int32 * n)(*codes)]
    return dev, n, arr


def _grad_workspace(n: int, dev, workspace):
    out = ctypes.c_size_t(0)
    B.check(B.load().flce_grad_norm_workspace_size(n, ctypes.byref(out)), "flce_grad_norm_workspace_size")
    return _workspace(out.value, dev, workspace), out.value


def grad_norm(grads: Iterable[torch.Tensor], *, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The 2-norm of all elements of all ``grads``, a 0-dim fp32 device tensor (see ``flce_grad_norm``)."""
    grads = list(grads)
    out = _call("clip_grad_norm", grads, None, None, workspace)
    if out is not None:
        return out[0]
    dev, n, (src, _, numel, codes) = _grad_arrays(grads, None)
    ws, nbytes = _grad_workspace(n, dev, workspace)
    norm = torch.empty((), dtype=torch.float32, device=dev)
    B.check(B.load().flce_grad_norm(src, numel, codes, n, norm.data_ptr(), ws.data_ptr(), nbytes, _stream(dev)),
            "flce_grad_norm")
    return norm


def clip_grad_norm_(grads: Iterable[torch.Tensor], max_norm: float, *,
                    outputs: Optional[Iterable[torch.Tensor]] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Scale ``grads`` by min(1, max_norm / (norm + 1e-6)) in place, or into ``outputs`` (tensors of the same
    dtypes and layouts, such as slices of an optimizer's flat buffer), and return the norm before clipping as a
    0-dim fp32 device tensor (see ``flce_clip_grad_norm``).  Nothing waits for the device.  List no gradient twice,
    and none that overlaps another: they are scaled side by side.  Nothing is recorded for autograd; what is written
    counts as changed in place, so that a backward that saved it raises."""
    grads = list(grads)
    outputs = None if outputs is None else list(outputs)
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError(f"flce: max_norm must not be negative, got {max_norm}")
    out = _call("clip_grad_norm", grads, max_norm, outputs, workspace)
    if out is not None:
        return out[0]
    dev, n, (src, dst, numel, codes) = _grad_arrays(grads, outputs)
    ws, nbytes = _grad_workspace(n, dev, workspace)
    norm = torch.empty((), dtype=torch.float32, device=dev)
    B.check(B.load().flce_clip_grad_norm(src, dst, numel, codes, n, max_norm, norm.data_ptr(), ws.data_ptr(), nbytes,
                                         _stream(dev)), "flce_clip_grad_norm")
    for t in grads if outputs is None else outputs:
        increment_version(t)
    return norm


# ---------------------------------------------------------------------------------------------------
# Penalties, biases and masks on logits
# ---------------------------------------------------------------------------------------------------
class ProcessedLogits(NamedTuple):
    logits: torch.Tensor  # [B, V]
    token: torch.Tensor   # [B] int64: greedy choice, -1 where nothing is allowed
    lse: torch.Tensor     # [B] fp32 log-sum-exp of the processed logits


@lru_cache(maxsize=256)
def _logits_problem(*fields):
    return B.FlceLogitsProblem(*fields)


def _per_request(t, b, dtype, name):
    if t is not None and (t.shape != (b,) or t.dtype != dtype or not t.is_contiguous()):
        raise ValueError(f"flce: {name} must be a contiguous {dtype} vector of {b} elements")


def _ids(t, b, name):
    if t.dim() != 2 or t.shape[0] != b or t.dtype not in (torch.int64, torch.int32):
        raise ValueError(f"flce: {name} must be an int64 or int32 matrix of {b} rows")
    return _rows(t, name)


def process_logits(logits: torch.Tensor, *, tokens: Optional[torch.Tensor] = None,
                   lens: Optional[torch.Tensor] = None, prompt_lens: Optional[torch.Tensor] = None,
                   repetition: Optional[torch.Tensor] = None, presence: Optional[torch.Tensor] = None,
                   frequency: Optional[torch.Tensor] = None, bias_ids: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                   workspace: Optional[torch.Tensor] = None) -> ProcessedLogits:
    """Penalties, biases and a mask on the logits [B, V] of B requests, with the greedy token and the
    log-sum-exp (see ``flce_process_logits`` in include/flce.h for the chain).

    ``tokens`` [B, H]: each request's history, of which the first ``lens[b]`` columns count and the first
    ``prompt_lens[b]`` are its prompt; ``repetition``, ``presence``, ``frequency`` [B] fp32.  ``bias_ids`` and
    ``bias`` [B, K]: sparse additions.  Ids outside [0, V) are padding.  ``mask`` [B, ceil(V / 32)] int32: bit
    v % 32 of word v // 32 allows entry v.  ``out`` may be ``logits``; ``out_dtype`` is logits' dtype or fp32.

    Nothing is recorded for autograd: the results carry no gradient, whatever the logits do, and a given ``out`` counts
    as changed in place, so that a backward that saved it raises."""
    res = _call("process_logits", logits, tokens, lens, prompt_lens, repetition, presence, frequency, bias_ids, bias,
                mask, out, -1 if out_dtype is None else _code(out_dtype, "out"), workspace)
    if res is not None:
        return ProcessedLogits._make(res)
    dev = logits.device
    _on(dev, logits=logits, tokens=tokens, lens=lens, prompt_lens=prompt_lens, repetition=repetition,
        presence=presence, frequency=frequency, bias_ids=bias_ids, bias=bias, mask=mask, out=out)
    if logits.dim() != 2 or logits.shape[1] == 0:
        raise ValueError("flce: logits must be a matrix with at least one column")
    logits = _rows(logits, "logits")
    b, v = logits.shape
    if tokens is None and not (lens is None and prompt_lens is None and repetition is None and presence is None
                               and frequency is None):
        raise ValueError("flce: lens, prompt_lens and the penalties need tokens")
    if (bias_ids is None) != (bias is None):
        raise ValueError("flce: bias_ids and bias go together")
    h = ts = k = bis = bs = ms = t64 = b64 = 0
    if tokens is not None:
        tokens = _ids(tokens, b, "tokens")
        h, ts, t64 = tokens.shape[1], tokens.stride(0), int(tokens.dtype == torch.int64)
        _per_request(lens, b, torch.int64, "lens")
        _per_request(prompt_lens, b, torch.int64, "prompt_lens")
        _per_request(repetition, b, torch.float32, "repetition")
        _per_request(presence, b, torch.float32, "presence")
        _per_request(frequency, b, torch.float32, "frequency")
    if bias is not None:
        bias_ids = _ids(bias_ids, b, "bias_ids")
        bias = _rows(bias, "bias")
        if bias.shape != bias_ids.shape or bias.dtype != torch.float32:
            raise ValueError("flce: bias must be fp32 with the shape of bias_ids")
        k, bis, bs, b64 = bias.shape[1], bias_ids.stride(0), bias.stride(0), int(bias_ids.dtype == torch.int64)
    if mask is not None:
        if mask.shape != (b, (v + 31) // 32) or mask.dtype != torch.int32:
            raise ValueError(f"flce: mask must be int32 of shape {(b, (v + 31) // 32)}")
        mask = _rows(mask, "mask")
        ms = mask.stride(0)
    given = out is not None
    if not given:
        out = torch.empty((b, v), dtype=out_dtype or logits.dtype, device=dev)
    elif out.shape != logits.shape or (out_dtype is not None and out.dtype != out_dtype) or \
            (v > 1 and out.stride(1) != 1):
        raise ValueError("flce: out must have logits' shape, out_dtype and adjacent elements in a row")
    prob = _logits_problem(b, v, h, k, logits.stride(0), out.stride(0), ts, bis, bs, ms,
                           _code(logits.dtype, "logits"), _code(out.dtype, "out"), t64, b64)
    token = torch.empty(b, dtype=torch.int64, device=dev)
    lse = torch.empty(b, dtype=torch.float32, device=dev)
    lib = B.load()
    size = ctypes.c_size_t(0)
    B.check(lib.flce_process_logits_workspace_size(ctypes.byref(prob), ctypes.byref(size)),
            "flce_process_logits_workspace_size")
    ws = _workspace(size.value, dev, workspace)
    if h == 0:
        tokens = lens = prompt_lens = repetition = presence = frequency = None
    if k == 0:
        bias_ids = bias = None
    B.check(lib.flce_process_logits(ctypes.byref(prob), _addr(logits), _addr(tokens), _addr(lens), _addr(prompt_lens),
                                    _addr(repetition), _addr(presence), _addr(frequency), _addr(bias_ids),
                                    _addr(bias), _addr(mask), _addr(out), _addr(token), _addr(lse), _addr(ws),
                                    size.value, _stream(dev)), "flce_process_logits")
    if given:
        increment_version(out)
    return ProcessedLogits(out, token, lse)
