"""The experts: what runs between dispatch and combine (``include/moe_route.h``, "The experts").

E4M3 tensors are uint8 codes with one power-of-two scale per block, float32 or uint8
(UE8M0) as dispatch writes them: [R, C/128] for rows, [E, ceil(rows/128), ceil(cols/128)]
for weights.  A training step of one layer's MLP::

    W1q, W1s = quantize_weight(W1)                     # after each optimizer step
    d  = dispatch(idx, E, X, fp8=True, bf16=False)
    h  = expert_swiglu(d.X_fp8, d.X_scale, W1q, W1s, d.expert_offsets)
    y  = expert_gemm(h.A_fp8, h.A_scale, W2q, W2s, d.expert_offsets)
    ...
    b   = expert_swiglu_backward(dY_fp8, dY_scale, W2q, W2s, h.GU_fp8, h.GU_scale, d.expert_offsets)
    dW2 = expert_wgrad(dY, h.A_fp8, h.A_scale, d.expert_offsets)
    dX  = expert_gemm(b.dGU_fp8, b.dGU_scale, W1q, W1s, d.expert_offsets, transpose=True)
    dW1 = expert_wgrad(b.dGU, d.X_fp8, d.X_scale, d.expert_offsets)

Kept from the forward to the backward pass: E4M3 rows only.  ``expert_swiglu`` is ``expert_gemm`` and ``swiglu`` in
one launch, ``expert_swiglu_backward`` the transposed ``expert_gemm`` and ``swiglu_backward``; what the single calls
round to bf16 between them stays in 32 bits there.  For serving a few tokens,
``moe_layer`` is the whole layer in one launch.

With ``stream`` a call launches there, and what it allocates is that stream's memory, as under
``torch.cuda.stream(stream)``; ordering it against other streams is the caller's.
"""
from __future__ import annotations

import functools
from dataclasses import dataclass
from typing import Optional

import torch

from . import _check, _need, _scale_dtype, _scale_format, _status_ptr, _workspace_arg, lib

__all__ = ["quantize_weight", "expert_gemm", "expert_wgrad", "swiglu", "swiglu_backward", "expert_swiglu",
           "expert_swiglu_backward", "moe_layer", "layer_workspace_size", "layer_workspace", "SwiGLU", "SwiGLUGrad", "LayerOut"]

BLOCK = 128


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _home(t: torch.Tensor, name: str) -> int:
    """The current device, which a call's first tensor has to be on."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        _need(t, name, t.dtype)
    return dev


def _arg(t: torch.Tensor, name: str, dtype, shape, dev: int) -> int:
    """The address of a tensor that _need accepts.  (These calls take up to a dozen tensors, and a small
    one's kernel runs for a few microseconds: what is right is found out in one expression.)"""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == dev):
        _need(t, name, dtype, shape)
    return t.data_ptr()


def _opt(t: Optional[torch.Tensor], name: str, dtype, shape, dev: int):
    return None if t is None else _arg(t, name, dtype, shape, dev)


def _scales(t: torch.Tensor, name: str, shape, dev: int):
    """The address of block scales of either format, and the format."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is torch.uint8:
        return _arg(t, name, torch.uint8, shape, dev), 1
    if t.dtype is not torch.float32:
        raise TypeError(f"{name} must be torch.float32 or torch.uint8 (UE8M0), got {t.dtype}")
    return _arg(t, name, torch.float32, shape, dev), 0


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """Memory for a result, of the stream that will write it: a block of the current stream may still be read by
    what is queued there, or be handed out again there, while another stream writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _on(stream, make, *args):
    """make(*args), what it allocates being the memory of `stream` (None: of the current one)."""
    if stream is None:
        return make(*args)
    with torch.cuda.stream(stream):
        return make(*args)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dims(t: torch.Tensor, name: str, n: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {tuple(t.shape)}")
    return tuple(t.shape)


def _groups(expert_offsets: Optional[torch.Tensor], E: Optional[int], dev: int):
    """The address of the offsets (or None), and the number of experts."""
    if expert_offsets is None:
        if E not in (None, 1):
            raise ValueError("expert_offsets is required for more than one expert")
        return None, 1
    if E is None:
        E = _dims(expert_offsets, "expert_offsets", 1)[0] - 1
    return _arg(expert_offsets, "expert_offsets", torch.int32, (E + 1,), dev), E


def quantize_weight(W: torch.Tensor, scale_format: str = "fp32", out=None, stream=None):
    """bf16 [E, rows, cols] (or [rows, cols]) -> (E4M3 codes uint8, scales of 128x128 blocks).
    `out`: the two tensors to write."""
    fmt = _scale_format(scale_format)
    if not isinstance(W, torch.Tensor) or W.dim() not in (2, 3):
        raise ValueError("W must be a tensor [E, rows, cols] or [rows, cols]")
    dev, whole = _home(W, "W"), W.shape
    src = _arg(W, "W", torch.bfloat16, whole, dev)
    E, rows, cols = whole if len(whole) == 3 else (1, *whole)
    shape = (E, _blocks(rows), _blocks(cols)) if len(whole) == 3 else (_blocks(rows), _blocks(cols))
    if out is None:
        q = _new(whole, torch.uint8, W.device, stream)
        s = _new(shape, _scale_dtype(scale_format), W.device, stream)
        qp, sp = q.data_ptr(), s.data_ptr()
    else:
        q, s = out
        qp = _arg(q, "W_fp8", torch.uint8, whole, dev)
        sp = _arg(s, "W_scale", _scale_dtype(scale_format), shape, dev)
    code = lib().moe_quantize_weight(src, E, rows, cols, qp, sp, fmt, _raw_stream(stream, dev))
    if code:
        _check(code, "moe_quantize_weight")
    return q, s


def expert_gemm(X_fp8: torch.Tensor, X_scale: torch.Tensor, W_fp8: torch.Tensor, W_scale: torch.Tensor,
                expert_offsets: Optional[torch.Tensor] = None, transpose: bool = False, out=None, status=None,
                stream=None) -> torch.Tensor:
    """Each expert's rows times its weight [rows, cols], bf16: x W^T, or x W with `transpose`
    (the gradient of the first one's input).  Without expert_offsets all rows are one group
    (W [1, rows, cols] or [rows, cols]).  Rows of no group are left as `out` has them."""
    if isinstance(W_fp8, torch.Tensor) and W_fp8.dim() == 2:
        W_fp8, W_scale = W_fp8[None], W_scale[None] if isinstance(W_scale, torch.Tensor) else W_scale
    E, rows, cols = _dims(W_fp8, "W_fp8", 3)
    R, red = _dims(X_fp8, "X_fp8", 2)
    if red != (rows if transpose else cols):
        raise ValueError(f"X_fp8 has {red} columns, W_fp8 {tuple(W_fp8.shape)} takes {rows if transpose else cols}")
    dev = _home(X_fp8, "X_fp8")
    x, w = _arg(X_fp8, "X_fp8", torch.uint8, (R, red), dev), _arg(W_fp8, "W_fp8", torch.uint8, (E, rows, cols), dev)
    xs, xf = _scales(X_scale, "X_scale", (R, red // BLOCK), dev)
    ws, wf = _scales(W_scale, "W_scale", (E, _blocks(rows), _blocks(cols)), dev)
    off, _ = _groups(expert_offsets, E, dev)
    n = cols if transpose else rows
    if out is None:
        out = _new((R, n), torch.bfloat16, X_fp8.device, stream)
        y = out.data_ptr()
    else:
        y = _arg(out, "out", torch.bfloat16, (R, n), dev)
    code = lib().moe_expert_gemm(x, xs, xf, w, ws, wf, off, R, E, rows, cols, int(bool(transpose)), y,
                                 _status_ptr(status), _raw_stream(stream, dev))
    if code:
        _check(code, "moe_expert_gemm")
    return out


def expert_wgrad(dY: torch.Tensor, X_fp8: torch.Tensor, X_scale: torch.Tensor,
                 expert_offsets: Optional[torch.Tensor] = None, dtype=torch.float32,
                 add: Optional[torch.Tensor] = None, out=None, status=None, stream=None) -> torch.Tensor:
    """Weight gradients [E, rows, cols] = add + dY^T x of each expert's rows, from the E4M3 rows that
    went into expert_gemm; dtype float32 or bfloat16.  `out` may be `add` (float32): the sum is then
    accumulated in place."""
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dtype must be torch.float32 or torch.bfloat16")
    R, rows = _dims(dY, "dY", 2)
    cols = _dims(X_fp8, "X_fp8", 2)[1]
    dev = _home(dY, "dY")
    dy, x = _arg(dY, "dY", torch.bfloat16, (R, rows), dev), _arg(X_fp8, "X_fp8", torch.uint8, (R, cols), dev)
    xs, xf = _scales(X_scale, "X_scale", (R, cols // BLOCK), dev)
    off, E = _groups(expert_offsets, None, dev)
    shape = (E, rows, cols)
    added = _opt(add, "add", torch.float32, shape, dev)
    if out is None:
        out = _new(shape, dtype, dY.device, stream)
    _check(lib().moe_expert_wgrad(dy, x, xs, xf, off, R, E, rows, cols, added, _arg(out, "out", dtype, shape, dev),
                                  int(dtype is torch.bfloat16), _status_ptr(status), _raw_stream(stream, dev)),
           "moe_expert_wgrad")
    return out


@dataclass
class SwiGLU:
    A_fp8: torch.Tensor
    A_scale: torch.Tensor
    GU_fp8: Optional[torch.Tensor] = None
    GU_scale: Optional[torch.Tensor] = None


@dataclass
class SwiGLUGrad:
    dGU: Optional[torch.Tensor]
    dGU_fp8: Optional[torch.Tensor]
    dGU_scale: Optional[torch.Tensor]


def _coded(R: int, C: int, scale_format: str, device, stream):
    return (_new((R, C), torch.uint8, device, stream),
            _new((R, C // BLOCK), _scale_dtype(scale_format), device, stream))


def swiglu(GU: torch.Tensor, keep: bool = True, scale_format: str = "fp32", out: Optional[SwiGLU] = None,
           stream=None) -> SwiGLU:
    """silu(gate) * up of GU bf16 [R, 2I] (gate columns first) in E4M3; with `keep` also GU in E4M3,
    which is all that swiglu_backward needs."""
    fmt = _scale_format(scale_format)
    R, C = _dims(GU, "GU", 2)
    dev = _home(GU, "GU")
    src = _arg(GU, "GU", torch.bfloat16, (R, C), dev)
    if C % (2 * BLOCK) != 0:
        raise ValueError("GU must be [R, 2I] with I a multiple of 128")
    I, sd = C // 2, _scale_dtype(scale_format)
    if out is None:
        out = SwiGLU(*_coded(R, I, scale_format, GU.device, stream),
                     *(_coded(R, C, scale_format, GU.device, stream) if keep else (None, None)))
    _check(lib().moe_swiglu(src, R, I, _arg(out.A_fp8, "A_fp8", torch.uint8, (R, I), dev),
                            _arg(out.A_scale, "A_scale", sd, (R, I // BLOCK), dev),
                            _opt(out.GU_fp8, "GU_fp8", torch.uint8, (R, C), dev),
                            _opt(out.GU_scale, "GU_scale", sd, (R, C // BLOCK), dev), fmt, _raw_stream(stream, dev)), "moe_swiglu")
    return out


def swiglu_backward(dA: torch.Tensor, GU_fp8: torch.Tensor, GU_scale: torch.Tensor, bf16: bool = True, fp8: bool = True,
                    scale_format: str = "fp32", out: Optional[SwiGLUGrad] = None, status=None,
                    stream=None) -> SwiGLUGrad:
    """Gradient of swiglu from its E4M3 checkpoint: dGU in bf16 (for expert_wgrad) and/or in E4M3 (for
    the transposed expert_gemm)."""
    fmt = _scale_format(scale_format)
    R, I = _dims(dA, "dA", 2)
    dev = _home(dA, "dA")
    da, kept = _arg(dA, "dA", torch.bfloat16, (R, I), dev), _arg(GU_fp8, "GU_fp8", torch.uint8, (R, 2 * I), dev)
    gs, gf = _scales(GU_scale, "GU_scale", (R, 2 * I // BLOCK), dev)
    if out is None:
        out = SwiGLUGrad(_new((R, 2 * I), torch.bfloat16, dA.device, stream) if bf16 else None,
                         *(_coded(R, 2 * I, scale_format, dA.device, stream) if fp8 else (None, None)))
    _check(lib().moe_swiglu_backward(da, kept, gs, gf, R, I, _opt(out.dGU, "dGU", torch.bfloat16, (R, 2 * I), dev),
                                     _opt(out.dGU_fp8, "dGU_fp8", torch.uint8, (R, 2 * I), dev),
                                     _opt(out.dGU_scale, "dGU_scale", _scale_dtype(scale_format), (R, 2 * I // BLOCK), dev),
                                     fmt, _status_ptr(status), _raw_stream(stream, dev)), "moe_swiglu_backward")
    return out


def _swiglu_out(R: int, I: int, keep: bool, sd, device) -> SwiGLU:
    e, u8 = torch.empty, torch.uint8
    return SwiGLU(e((R, I), dtype=u8, device=device), e((R, I // BLOCK), dtype=sd, device=device),
                  e((R, 2 * I), dtype=u8, device=device) if keep else None,
                  e((R, 2 * I // BLOCK), dtype=sd, device=device) if keep else None)


def _swiglu_grad_out(R: int, I: int, bf16: bool, fp8: bool, sd, device) -> SwiGLUGrad:
    e = torch.empty
    return SwiGLUGrad(e((R, 2 * I), dtype=torch.bfloat16, device=device) if bf16 else None,
                      e((R, 2 * I), dtype=torch.uint8, device=device) if fp8 else None,
                      e((R, 2 * I // BLOCK), dtype=sd, device=device) if fp8 else None)


def _joined(X_fp8, X_scale, W_fp8, W_scale, expert_offsets, names, backward):
    """The arguments that expert_swiglu and its gradient share: (device, addresses and formats, R, E, H, I)."""
    x_name, w_name = names
    if isinstance(W_fp8, torch.Tensor) and W_fp8.dim() == 2:
        W_fp8, W_scale = W_fp8[None], W_scale[None] if isinstance(W_scale, torch.Tensor) else W_scale
    E, rows, cols = _dims(W_fp8, w_name + "_fp8", 3)
    R, H = _dims(X_fp8, x_name + "_fp8", 2)
    if H != (rows if backward else cols):
        raise ValueError(f"{x_name}_fp8 has {H} columns, {w_name}_fp8 {tuple(W_fp8.shape)} takes {rows if backward else cols}")
    I = cols if backward else rows // 2
    if H % BLOCK != 0 or I % BLOCK != 0 or (not backward and rows % 2 != 0):
        raise ValueError(f"{w_name}_fp8 must be [E, {'H, I' if backward else '2I, H'}] with H and I multiples of 128")
    dev = _home(X_fp8, x_name + "_fp8")
    x = _arg(X_fp8, x_name + "_fp8", torch.uint8, (R, H), dev)
    xs, xf = _scales(X_scale, x_name + "_scale", (R, H // BLOCK), dev)
    w = _arg(W_fp8, w_name + "_fp8", torch.uint8, (E, rows, cols), dev)
    ws, wf = _scales(W_scale, w_name + "_scale", (E, rows // BLOCK, cols // BLOCK), dev)
    off, _ = _groups(expert_offsets, E, dev)
    return dev, (x, xs, xf, w, ws, wf, off), R, E, H, I


def expert_swiglu(X_fp8: torch.Tensor, X_scale: torch.Tensor, W1_fp8: torch.Tensor, W1_scale: torch.Tensor,
                  expert_offsets: Optional[torch.Tensor] = None, keep: bool = True, scale_format: str = "fp32",
                  out: Optional[SwiGLU] = None, status=None, stream=None) -> SwiGLU:
    """swiglu(expert_gemm(X, W1)) in one launch, without the bf16 rows between: W1 [E, 2I, H] (gate rows first)
    or [2I, H].  With `keep` also the products in E4M3, for expert_swiglu_backward or swiglu_backward.  Rows of
    no group are left as `out` has them."""
    fmt, sd = _scale_format(scale_format), _scale_dtype(scale_format)
    dev, args, R, E, H, I = _joined(X_fp8, X_scale, W1_fp8, W1_scale, expert_offsets, ("X", "W1"), False)
    if out is None:
        out = _on(stream, _swiglu_out, R, I, keep, sd, X_fp8.device)
        a, sa, k, sk = out.A_fp8.data_ptr(), out.A_scale.data_ptr(), _ptr(out.GU_fp8), _ptr(out.GU_scale)
    else:
        a, sa = _arg(out.A_fp8, "A_fp8", torch.uint8, (R, I), dev), _arg(out.A_scale, "A_scale", sd, (R, I // BLOCK), dev)
        k = _opt(out.GU_fp8, "GU_fp8", torch.uint8, (R, 2 * I), dev)
        sk = _opt(out.GU_scale, "GU_scale", sd, (R, 2 * I // BLOCK), dev)
    code = lib().moe_expert_swiglu(*args, R, E, H, I, a, sa, k, sk, fmt, _status_ptr(status), _raw_stream(stream, dev))
    if code:
        _check(code, "moe_expert_swiglu")
    return out


def expert_swiglu_backward(dY_fp8: torch.Tensor, dY_scale: torch.Tensor, W2_fp8: torch.Tensor, W2_scale: torch.Tensor,
                           GU_fp8: torch.Tensor, GU_scale: torch.Tensor, expert_offsets: Optional[torch.Tensor] = None,
                           bf16: bool = True, fp8: bool = True, scale_format: str = "fp32",
                           out: Optional[SwiGLUGrad] = None, status=None, stream=None) -> SwiGLUGrad:
    """swiglu_backward(expert_gemm(dY, W2, transpose=True), GU) in one launch, without the bf16 rows between:
    W2 [E, H, I] or [H, I]; dGU in bf16 (for expert_wgrad) and/or in E4M3 (for the transposed expert_gemm)."""
    fmt = _scale_format(scale_format)
    dev, args, R, E, H, I = _joined(dY_fp8, dY_scale, W2_fp8, W2_scale, expert_offsets, ("dY", "W2"), True)
    kept = _arg(GU_fp8, "GU_fp8", torch.uint8, (R, 2 * I), dev)
    gs, gf = _scales(GU_scale, "GU_scale", (R, 2 * I // BLOCK), dev)
    sd = _scale_dtype(scale_format)
    if out is None:
        out = _on(stream, _swiglu_grad_out, R, I, bf16, fp8, sd, dY_fp8.device)
        d, q, sq = _ptr(out.dGU), _ptr(out.dGU_fp8), _ptr(out.dGU_scale)
    else:
        d = _opt(out.dGU, "dGU", torch.bfloat16, (R, 2 * I), dev)
        q = _opt(out.dGU_fp8, "dGU_fp8", torch.uint8, (R, 2 * I), dev)
        sq = _opt(out.dGU_scale, "dGU_scale", sd, (R, 2 * I // BLOCK), dev)
    code = lib().moe_expert_swiglu_backward(*args, kept, gs, gf, R, E, H, I, d, q, sq, fmt, _status_ptr(status),
                                            _raw_stream(stream, dev))
    if code:
        _check(code, "moe_expert_swiglu_backward")
    return out


@dataclass
class LayerOut:
    out: torch.Tensor
    topk_idx: torch.Tensor
    topk_w: torch.Tensor


_layer_workspaces = {}


@functools.lru_cache(maxsize=None)
def layer_workspace_size(N: int, H: int, I: int, E: int, K: int) -> int:
    """Bytes of workspace moe_layer needs (0 for sizes it does not take)."""
    return int(lib().moe_layer_workspace_size(N, H, I, E, K))


def _capturing(stream) -> bool:
    """Whether a CUDA graph is being captured on `stream` (None: the current one)."""
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def layer_workspace(N: int, H: int, I: int, E: int, K: int, device=None, stream=None) -> torch.Tensor:
    """A workspace for moe_layer, cached per (device, stream, E, I) and grown where a call needs more.
    Its counters start at zero and every call leaves them there, so one buffer serves all calls of one
    stream; calls that may overlap on the GPU must not share it.

    While a graph is being captured on the stream the buffer is a new one of the capture's own memory, its
    counters cleared by the graph, and the cache is left alone: graphs may be replayed in any order and next
    to plain calls, and what a graph holds is neither shared with a later call nor freed when one needs more.
    (A buffer taken outside and passed to a captured call is the graph's for as long as the graph is used.)"""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if stream is None:
        stream = torch.cuda.current_stream(device)
    need = layer_workspace_size(N, H, I, E, K)
    if _capturing(stream):
        with torch.cuda.stream(stream):
            ws = torch.empty(need, dtype=torch.uint8, device=device)
            ws[:256 + 4 * (E + 128) * (I // BLOCK)].zero_()     # what moe_route.h asks to be zero
        return ws
    key = (device.index, stream.cuda_stream, E, I)
    ws = _layer_workspaces.get(key)
    if ws is None or ws.numel() < need:
        with torch.cuda.stream(stream):
            ws = torch.zeros(need, dtype=torch.uint8, device=device)
        _layer_workspaces[key] = ws
    return ws


def moe_layer(X: torch.Tensor, W_gate: torch.Tensor, K: int, W1_fp8: torch.Tensor, W1_scale: torch.Tensor,
              W2_fp8: torch.Tensor, W2_scale: torch.Tensor, bias: Optional[torch.Tensor] = None, renorm: bool = True,
              residual: Optional[torch.Tensor] = None, out: Optional[LayerOut] = None,
              workspace: Optional[torch.Tensor] = None, status=None, stream=None) -> LayerOut:
    """The whole layer (router, gated MLP of the K chosen experts, weighted sum, residual) for up to 64
    tokens in one launch.  W1 [E, 2I, H] (gate rows first) and W2 [E, H, I] in E4M3 with 128x128 scales
    of one format (quantize_weight); X bf16 [N, H].  `out.out` may be the residual."""
    N, H = _dims(X, "X", 2)
    E, two_i, _ = _dims(W1_fp8, "W1_fp8", 3)
    I = two_i // 2
    dev = _home(X, "X")
    x, wg = _arg(X, "X", torch.bfloat16, (N, H), dev), _arg(W_gate, "W_gate", torch.bfloat16, (H, E), dev)
    w1, w2 = _arg(W1_fp8, "W1_fp8", torch.uint8, (E, 2 * I, H), dev), _arg(W2_fp8, "W2_fp8", torch.uint8, (E, H, I), dev)
    s1, fmt = _scales(W1_scale, "W1_scale", (E, _blocks(2 * I), _blocks(H)), dev)
    s2, fmt2 = _scales(W2_scale, "W2_scale", (E, _blocks(H), _blocks(I)), dev)
    if fmt2 != fmt:
        raise TypeError("W1_scale and W2_scale must be of one format")
    b, res = _opt(bias, "bias", torch.float32, (E,), dev), _opt(residual, "residual", torch.bfloat16, (N, H), dev)
    if out is None:
        out = LayerOut(_new((N, H), torch.bfloat16, X.device, stream), _new((N, K), torch.int32, X.device, stream),
                       _new((N, K), torch.float32, X.device, stream))
    raw = _raw_stream(stream, dev)
    if workspace is not None:
        ws, ws_bytes = _workspace_arg(workspace)
    elif layer_workspace_size(N, H, I, E, K):
        cached = None if _capturing(stream) else _layer_workspaces.get((dev, raw, E, I))
        if cached is None or cached.numel() < layer_workspace_size(N, H, I, E, K):
            cached = layer_workspace(N, H, I, E, K, X.device, stream)
        ws, ws_bytes = cached.data_ptr(), cached.numel()
    else:
        ws, ws_bytes = None, 0
    _check(lib().moe_layer(x, wg, b, w1, s1, w2, s2, fmt, res, N, H, I, E, K, int(bool(renorm)),
                           _arg(out.topk_idx, "topk_idx", torch.int32, (N, K), dev),
                           _arg(out.topk_w, "topk_w", torch.float32, (N, K), dev),
                           _arg(out.out, "out", torch.bfloat16, (N, H), dev), _status_ptr(status), ws, ws_bytes, raw),
           "moe_layer")
    return out
