"""The norms around the experts (``include/moe_route.h``, "The norms around the experts"): the RMS norm in front
of the router with the residual stream's addition, and the norm of all gradients with its clipping.

A block and its training step::

    n   = rms_norm(attn, w, residual=x)              # n.S is the stream, n.Y what the router reads
    idx, rw, d, _ = route_dispatch(n.Y, W_gate, K)
    ...                                              # the experts: see experts.py
    out = combine(y, d.row_map, rw, residual=n.S)
    ...
    g = rms_norm_backward(dY, n.S, w, n.rstd, dS=dout)   # dout: out's gradient, through the stream
    clip_grad_norm([dW1, dW2, g.dweight], 1.0)

With ``stream`` a call launches there, and what it allocates is that stream's memory, as in experts.py.
"""
from __future__ import annotations

from array import array
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import _check, _need, _scale_dtype, _scale_format, _status_ptr, lib
from .experts import BLOCK, _arg, _dims, _home, _on, _opt, _ptr, _raw_stream

__all__ = ["rms_norm", "rms_norm_backward", "grad_norm", "clip_grad_norm", "RMSNorm", "RMSNormGrad"]

_TYPES = {torch.float32: 0, torch.bfloat16: 1}


def _weight(w: torch.Tensor, H: int, dev: int):
    """The address of a weight of either type, and the type."""
    if not isinstance(w, torch.Tensor):
        raise TypeError("weight must be a torch.Tensor")
    if w.dtype not in _TYPES:
        raise TypeError(f"weight must be torch.float32 or torch.bfloat16, got {w.dtype}")
    return _arg(w, "weight", w.dtype, (H,), dev), _TYPES[w.dtype]


@dataclass
class RMSNorm:
    Y: Optional[torch.Tensor]
    Y_fp8: Optional[torch.Tensor]
    Y_scale: Optional[torch.Tensor]
    S: torch.Tensor
    rstd: Optional[torch.Tensor]


@dataclass
class RMSNormGrad:
    dX: torch.Tensor
    dweight: torch.Tensor


def _rms_out(X: torch.Tensor, N: int, H: int, stream_too: bool, bf16: bool, fp8: bool, sd) -> RMSNorm:
    e, device = torch.empty, X.device
    return RMSNorm(torch.empty_like(X) if bf16 else None,
                   e((N, H), dtype=torch.uint8, device=device) if fp8 else None,
                   e((N, H // BLOCK), dtype=sd, device=device) if fp8 else None,
                   torch.empty_like(X) if stream_too else X, e((N,), dtype=torch.float32, device=device))


def rms_norm(X: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             bf16: bool = True, fp8: bool = False, scale_format: str = "fp32", out: Optional[RMSNorm] = None,
             stream=None) -> RMSNorm:
    """y = s * rstd * weight with s = bf16(X + residual) (S; X itself without a residual) and rstd = 1 / sqrt(mean
    s^2 + eps): in bf16 (Y) and/or in E4M3 with 1x128 scales (Y_fp8, Y_scale).  X, residual bf16 [N, H], weight [H]
    float32 or bfloat16.  `out` names the tensors to write (None: not wanted; its S may be the residual, or X where Y
is not; without a residual it is X or None)."""
    fmt = _scale_format(scale_format)
    N, H = _dims(X, "X", 2)
    dev = _home(X, "X")
    x, res = _arg(X, "X", torch.bfloat16, (N, H), dev), _opt(residual, "residual", torch.bfloat16, (N, H), dev)
    w, wt = _weight(weight, H, dev)
    if out is None:
        if fp8 and H % BLOCK != 0:
            raise ValueError("E4M3 rows need H to be a multiple of 128")
        out = _on(stream, _rms_out, X, N, H, residual is not None, bf16, fp8, _scale_dtype(scale_format))
        y, q, sq, r = _ptr(out.Y), _ptr(out.Y_fp8), _ptr(out.Y_scale), out.rstd.data_ptr()
        s = None if residual is None else out.S.data_ptr()
    else:
        y, q = _opt(out.Y, "Y", torch.bfloat16, (N, H), dev), _opt(out.Y_fp8, "Y_fp8", torch.uint8, (N, H), dev)
        sq = _opt(out.Y_scale, "Y_scale", _scale_dtype(scale_format), (N, H // BLOCK), dev)
        r = _opt(out.rstd, "rstd", torch.float32, (N,), dev)
        if residual is not None:
            s = _arg(out.S, "S", torch.bfloat16, (N, H), dev)
        else:
            s = None
            if out.S is not None and out.S.data_ptr() != x:
                raise ValueError("without a residual the stream is X itself: S of `out` must be X or None")
    code = lib().moe_rms_norm(x, res, w, wt, eps, N, H, s, y, q, sq, fmt, r, _raw_stream(stream, dev))
    if code:
        _check(code, "moe_rms_norm")
    return out


def _rms_grad_out(dY: torch.Tensor, H: int, need: int, results: bool):
    device = dY.device
    return (RMSNormGrad(torch.empty_like(dY), torch.empty((H,), dtype=torch.float32, device=device)) if results else None,
            torch.empty((need,), dtype=torch.uint8, device=device))


def rms_norm_backward(dY: torch.Tensor, S: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                      dS: Optional[torch.Tensor] = None, add: Optional[torch.Tensor] = None,
                      out: Optional[RMSNormGrad] = None, status=None, stream=None) -> RMSNormGrad:
    """Gradient of rms_norm from its S and rstd: dX (of X and of the residual alike; dS, the gradient that reaches S
    through the stream, is added) and dweight float32 [H] = add + the sum over the rows."""
    N, H = _dims(dY, "dY", 2)
    dev = _home(dY, "dY")
    dy, s = _arg(dY, "dY", torch.bfloat16, (N, H), dev), _arg(S, "S", torch.bfloat16, (N, H), dev)
    w, wt = _weight(weight, H, dev)
    r, ds = _arg(rstd, "rstd", torch.float32, (N,), dev), _opt(dS, "dS", torch.bfloat16, (N, H), dev)
    added = _opt(add, "add", torch.float32, (H,), dev)
    need = lib().moe_rms_norm_backward_workspace_size(N, H)
    new, ws = _on(stream, _rms_grad_out, dY, H, need, out is None)
    if out is None:
        out, dx, dw = new, new.dX.data_ptr(), new.dweight.data_ptr()
    else:
        dx, dw = _arg(out.dX, "dX", torch.bfloat16, (N, H), dev), _arg(out.dweight, "dweight", torch.float32, (H,), dev)
    code = lib().moe_rms_norm_backward(dy, s, w, wt, r, ds, added, N, H, dx, dw, _status_ptr(status), ws.data_ptr(), need,
                                       _raw_stream(stream, dev))
    if code:
        _check(code, "moe_rms_norm_backward")
    return out


def _list(tensors: Sequence[torch.Tensor], name: str, dev: int):
    """(addresses, sizes, dtypes) of a list of tensors on the current device."""
    try:
        where = set(map(torch.Tensor.get_device, tensors))
        flat = all(map(torch.Tensor.is_contiguous, tensors))
        ptrs, sizes, dtypes = list(map(torch.Tensor.data_ptr, tensors)), list(map(torch.Tensor.numel, tensors)), [t.dtype for t in tensors]
    except TypeError:
        raise TypeError(f"{name} must be a list of torch.Tensors") from None
    if not (flat and where <= {dev} and _TYPES.keys() >= set(dtypes)):
        for i, t in enumerate(tensors):
            if t.dtype not in _TYPES:
                raise TypeError(f"{name}[{i}] must be torch.float32 or torch.bfloat16, got {t.dtype}")
            _need(t, f"{name}[{i}]", t.dtype)
    return ptrs, sizes, dtypes


def _distinct(ptrs, written, sizes):
    """Refuses a tensor that would be scaled twice, or into another one that is still to be read."""
    pairs = [(p, q) for p, q, k in zip(ptrs, written, sizes) if k]
    if len({q for _, q in pairs}) != len(pairs):
        raise ValueError("a tensor is listed twice: it would be scaled twice")
    read = {p for p, _ in pairs}
    if any(p != q and q in read for p, q in pairs):
        raise ValueError("out[i] may be grads[i], but no other of the gradients")


def _norm_out(need: int, device, result: bool):
    return (torch.empty((1,), dtype=torch.float32, device=device) if result else None,
            torch.empty((need,), dtype=torch.uint8, device=device))


def _norm_call(grads, out, max_norm, norm, stream):
    grads = list(grads)
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -2
    ptrs, sizes, dtypes = _list(grads, "grads", dev)
    if dev < 0:
        raise ValueError("gradients must be CUDA tensors (the library has no CPU path)")
    n = len(grads)
    written = ptrs
    if out is not None:
        out = list(out)
        written, out_sizes, out_dtypes = _list(out, "out", dev)
        if out_sizes != sizes or out_dtypes != dtypes:
            raise ValueError("out must have the sizes and types of grads")
    if max_norm is not None and len(set(ptrs if out is None else ptrs + written)) != (n if out is None else 2 * n):
        _distinct(ptrs, written, sizes)
    need = lib().moe_grad_norm_workspace_size(n)
    new, ws = _on(stream, _norm_out, need, torch.device("cuda", dev), norm is None)
    res = new.data_ptr() if norm is None else _arg(norm, "norm", torch.float32, (1,), dev)
    # (the arrays live until the call is over: the library reads them during the call only)
    src, count, types = array("Q", ptrs), array("q", sizes), array("i", map(_TYPES.__getitem__, dtypes))
    lists, raw = (src.buffer_info()[0], count.buffer_info()[0], types.buffer_info()[0]), _raw_stream(stream, dev)
    if max_norm is None:
        code = lib().moe_grad_norm(*lists, n, res, ws.data_ptr(), need, raw)
    else:
        dst = None if out is None else array("Q", written)
        code = lib().moe_clip_grad_norm(lists[0], None if dst is None else dst.buffer_info()[0], *lists[1:], n, max_norm,
                                        res, ws.data_ptr(), need, raw)
    if code:
        _check(code, "moe_grad_norm" if max_norm is None else "moe_clip_grad_norm")
    return new if norm is None else norm


def grad_norm(grads: Sequence[torch.Tensor], out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The 2-norm of a list of float32 and bfloat16 tensors together, float32 [1] on the device."""
    return _norm_call(grads, None, None, out, stream)


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, out: Optional[Sequence[torch.Tensor]] = None,
                   norm: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scale the tensors by min(1, max_norm / (norm + 1e-6)), in place or into the tensors of `out`, without the
    host seeing the norm; returns it (before the scaling), float32 [1].  If it is not finite, the tensors are left
    as they are (copied to `out`).  out[i] may be grads[i]; no tensor that is written may overlap another otherwise."""
    max_norm = float(max_norm)
    if not max_norm >= 0:
        raise ValueError("max_norm must not be negative or NaN")
    return _norm_call(grads, out, max_norm, norm, stream)
