"""The operators around and inside an expert block that join products with what follows them: what a pass computes and costs.

  rms_norm      the norm in front of the router: the residual stream's addition, root-mean-square norm with a weight, out in
                bf16 (what the router and the dispatch read) and, for a shared expert, in E4M3 with 1x128 scales; `backward`
                its gradient, with the residual stream's own gradient added and the weight's gradient summed over the tokens
  swiglu        the experts' gate and up projections, the activation and the product in one kernel: E4M3 rows in, E4M3 rows
                out, the checkpoint of both halves in E4M3; `backward` the input gradient of the down projection joined with
                the activation's gradient
  clip          the norm of all gradients of a model's expert blocks, and the gradients scaled down to a largest norm

`run` computes them in plain torch operations where `own` is false and through the package where it is true; `exact`
computes them in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLK = 128
EPS = 1e-6
E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
RCP448 = float(np.float32(1) / np.float32(448))


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # decoding one sequence: the norm is its own latency, its rows go to the router and to a shared expert
        dict(name="rms_norm_1tok_h2048", op="rms_norm", backward=False, N=1, H=2048, residual=True, fp8=True, weight="bf16"),
        # a training step of 65536 tokens
        dict(name="rms_norm_65536x4096", op="rms_norm", backward=False, N=65536, H=4096, residual=True, fp8=True, weight="fp32"),
        # gradient of an odd number of tokens of an odd width, the norm of a block without a residual stream
        dict(name="rms_norm_bwd_16381x1032", op="rms_norm", backward=True, N=16381, H=1032, residual=False, add=True, weight="fp32"),
        # gradient of the 65536-token step
        dict(name="rms_norm_bwd_65536x4096", op="rms_norm", backward=True, N=65536, H=4096, residual=True, add=False, weight="bf16"),
        # 65 tokens of a small layer: several experts hold one row or none, the call is its own latency
        dict(name="swiglu_65tok_e16", op="swiglu", backward=False, N=65, E=16, K=2, H=256, I=256, skew=0.0, keep=True, fmt="fp32"),
        # the training step of 16384 tokens, 128 experts, top 8
        dict(name="swiglu_16384tok_e128", op="swiglu", backward=False, N=16384, E=128, K=8, H=2048, I=1024, skew=0.0, keep=True, fmt="ue8m0"),
        # serving an odd number of tokens under an uneven load: no checkpoint
        dict(name="swiglu_serve_16381tok_e64", op="swiglu", backward=False, N=16381, E=64, K=2, H=1024, I=2048, skew=0.5, keep=False, fmt="fp32"),
        # gradient of a small step, some experts without rows
        dict(name="swiglu_bwd_1023tok_e64", op="swiglu", backward=True, N=1023, E=64, K=2, H=1024, I=512, skew=1.0, fmt="fp32"),
        # gradient of the 16384-token step
        dict(name="swiglu_bwd_16384tok_e128", op="swiglu", backward=True, N=16384, E=128, K=8, H=2048, I=1024, skew=0.0, fmt="ue8m0"),
        # the gradients of one small block, over the bound
        dict(name="clip_e4_h256", op="clip", L=1, E=4, H=256, I=128, grads="fp32", flat=False, clip=True, bound=0.3),
        # 24 small blocks of odd sizes whose bf16 gradients lie one behind the other in a buffer
        dict(name="clip_24_layers_odd", op="clip", L=24, E=8, H=511, I=257, grads="bf16", flat=True, clip=True, bound=0.9),
        # one block of the 16384-token step with half of its experts here, over the bound
        dict(name="clip_e64_h2048", op="clip", L=1, E=64, H=2048, I=1024, grads="fp32", flat=False, clip=True, bound=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi, step):
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    while True:
        op = rng.choice(["rms_norm", "swiglu", "swiglu", "clip"])
        backward = rng.random() < 0.5
        if op == "rms_norm":
            fp8 = not backward and rng.random() < 0.5
            c = dict(op=op, backward=backward, N=_log(rng, 1, 65536), H=_dim(rng, 128, 16384, 128) if fp8 else _dim(rng, 8, 16384, 8),
                     residual=rng.random() < 0.5, weight=rng.choice(["fp32", "bf16"]))
            c.update(add=rng.random() < 0.5) if backward else c.update(fp8=fp8)
            if c["N"] * c["H"] > 65536 * 4096:
                continue
        elif op == "swiglu":
            E = rng.choice([1, 5, 16, 64, 128])
            c = dict(op=op, backward=backward, N=_log(rng, 1, 16384), E=E, K=min(E, rng.choice([1, 2, 4, 8])), H=_dim(rng, 128, 4096, 128),
                     I=_dim(rng, 128, 2048, 128), skew=rng.choice([0.0, 0.5, 1.0]), fmt=rng.choice(["fp32", "ue8m0"]))
            if not backward:
                c["keep"] = rng.random() < 0.7
            # the plain form pads every group to the largest
            if c["N"] * c["K"] * c["H"] * c["I"] > 131072 * 2048 * 1024:
                continue
            if c["skew"] and (c["N"] * c["K"] > 32768 or c["N"] * E * max(c["H"], 2 * c["I"]) > 1 << 32):
                continue
        else:
            flat = rng.random() < 0.5
            c = dict(op=op, L=_log(rng, 1, 24 if flat else 12), E=rng.choice([1, 4, 16, 64]), H=_log(rng, 128, 2048), I=_log(rng, 128, 1024),
                     grads=rng.choice(["fp32", "bf16"]), flat=flat, clip=rng.random() < 0.7, bound=rng.choice([0.1, 0.9, 3.0]))
            if _elements(c) > 64 * 2048 * 1024 * 3:
                continue
        return c


def _touched(c):
    """Experts that N tokens of K distinct experts reach, on average."""
    return c["E"] * (1 - (1 - c["K"] / c["E"]) ** c["N"])


def _shapes(c):
    """The gradients of L blocks: both expert weights, the router's, the norm's."""
    E, H, I = c["E"], c["H"], c["I"]
    return [s for _ in range(c["L"]) for s in ((E, 2 * I, H), (E, H, I), (H, E), (H,))]


def _elements(c):
    return sum(math.prod(s) for s in _shapes(c))


def work(c):
    if c["op"] == "rms_norm":
        n, wb = c["N"] * c["H"], 2 if c["weight"] == "bf16" else 4
        if c["backward"]:   # dY, S in; dX out; the stream's gradient and what the weight's is added to
            return {"bytes": n * (6 + 2 * c["residual"]) + 4 * c["N"] + c["H"] * (wb + 4 + 4 * c["add"]), "flops": 10 * n}
        return {"bytes": n * (4 + 4 * c["residual"] + c["fp8"]) + (n // BLK if c["fp8"] else 0) + 4 * c["N"] + c["H"] * wb, "flops": 5 * n}
    if c["op"] == "swiglu":
        R, H, I, sb = c["N"] * c["K"], c["H"], c["I"], 1 if c["fmt"] == "ue8m0" else 4
        rows = R * (H + sb * H // BLK) + 4 * (c["E"] + 1)
        if c["backward"]:   # dY, W2, the checkpoint; dGU in bf16 and E4M3
            weights = _touched(c) * (H * I + sb * (H // BLK) * (I // BLK))
            return {"bytes": rows + weights + R * 2 * (I + sb * I // BLK) + R * 4 * I + R * 2 * (I + I // BLK), "flops": 2 * R * H * I + 20 * R * I}
        weights = _touched(c) * (2 * I * H + sb * 2 * (H // BLK) * (I // BLK))
        return {"bytes": rows + weights + R * (3 if c["keep"] else 1) * (I + I // BLK), "flops": 4 * R * H * I + 10 * R * I}
    e = sum(math.prod(s) * (2 if c["grads"] == "bf16" and len(s) == 3 else 4) for s in _shapes(c))
    return {"bytes": e * (1 + c["clip"]) + 4, "flops": _elements(c) * (2 + c["clip"])}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) + 2000003)


def _pow2ceil(t):
    """The power of two at or above t (fp32, positive), and 127 + its logarithm."""
    m, e = torch.frexp(t)
    e = torch.where(m == 0.5, e - 1, e) + 127
    return (e << 23).view(torch.float32), e


def _scale_out(s, e, fmt):
    return e.to(torch.uint8) if fmt == "ue8m0" else s


def _scale_in(scale):
    if scale.dtype == torch.uint8:
        return (scale.to(torch.int32) << 23).view(torch.float32)
    return scale


def _quant_rows(x, fmt):
    """fp32 [R, C] -> E4M3 codes (uint8) and scales of 1x128 blocks."""
    b = x.view(x.shape[0], -1, BLK)
    s, e = _pow2ceil(b.abs().amax(-1).clamp_min(1e-4) * RCP448)
    q = (b / s[..., None]).to(E4M3).view(x.shape)
    return q.view(torch.uint8), _scale_out(s, e, fmt)


def _quant_weight(W, fmt):
    """[E, n, k] -> E4M3 codes (uint8) and scales of 128x128 blocks; n and k are whole in 128."""
    E, n, k = W.shape
    b = W.view(E, n // BLK, BLK, k // BLK, BLK)
    s, e = _pow2ceil(b.abs().amax((2, 4)).float().clamp_min(1e-4) * RCP448)
    q = (b.float() / s[:, :, None, :, None]).to(E4M3).view(W.shape)
    return q.view(torch.uint8), _scale_out(s, e, fmt)


def _offsets(c, g):
    """Rows of each expert: every token takes K different experts, by a preference when the load is skewed."""
    pref = torch.rand((c["N"], c["E"]), generator=g, device=DEV).log().neg().log().neg()
    pref -= c["skew"] * torch.arange(1, c["E"] + 1, device=DEV).log()
    idx = pref.topk(c["K"], dim=1).indices
    off = torch.zeros(c["E"] + 1, dtype=torch.int32, device=DEV)
    off[1:] = torch.bincount(idx.flatten(), minlength=c["E"]).cumsum(0)
    return off


def _views(flat, c, kinds):
    """The gradients as views, one behind the other, of a buffer for each type."""
    at, out = {k: 0 for k in kinds}, []
    for sh, k in zip(_shapes(c), kinds):
        n = math.prod(sh)
        out.append(flat[k][at[k]:at[k] + n].view(sh))
        at[k] += n
    return out


def _joined(s, grads):
    """What a pass returns of the clipped gradients: the tensors, or the buffers that hold them one behind the other."""
    if not s["flat"]:
        return grads
    return [torch.cat([g.flatten() for t, g in zip(s["grads"], grads) if t.dtype is k]) for k in s["buffers"]]


def prepare(c, seed):
    g = _gen(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    s = dict(c)
    if c["op"] == "rms_norm":
        N, H = c["N"], c["H"]
        wt = torch.bfloat16 if c["weight"] == "bf16" else torch.float32
        s["w"] = (1 + normal(H, std=0.2, dtype=torch.float32)).to(wt)
        # a residual stream: every token has a length of its own, and a few channels are far larger than the rest
        size = torch.exp(normal(N, 1, dtype=torch.float32)) * torch.where(torch.rand(H, generator=g, device=DEV) < 0.01, 20.0, 1.0)
        x = (normal(N, H, dtype=torch.float32) * size).to(torch.bfloat16)
        if c["backward"]:
            s["S"], s["dY"] = x, normal(N, H, std=1e-2)
            s["rstd"] = torch.rsqrt(x.float().square().mean(1) + EPS)
            s["dS"] = normal(N, H, std=1e-2) if c["residual"] else None
            s["add"] = normal(H, dtype=torch.float32) if c["add"] else None
        else:
            s["X"] = normal(N, H) if c["residual"] else x
            s["res"] = x if c["residual"] else None
    elif c["op"] == "swiglu":
        s["offsets"] = _offsets(c, g)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        R, H, I, E = c["N"] * c["K"], c["H"], c["I"], c["E"]
        s["X"], s["X_scale"] = _quant_rows(normal(R, H, std=1e-2 if c["backward"] else 1.0).float(), c["fmt"])
        if c["backward"]:
            s["W"], s["W_scale"] = _quant_weight(normal(E, H, I, std=I ** -0.5), c["fmt"])
            s["GU"], s["GU_scale"] = _quant_rows(normal(R, 2 * I).float(), c["fmt"])
        else:
            s["W"], s["W_scale"] = _quant_weight(normal(E, 2 * I, H, std=H ** -0.5), c["fmt"])
    else:
        kinds = [torch.bfloat16 if c["grads"] == "bf16" and len(sh) == 3 else torch.float32 for sh in _shapes(c)]
        sizes = [math.prod(sh) for sh in _shapes(c)]
        std = 1e-3
        s["max_norm"] = c["bound"] * std * math.sqrt(sum(sizes))
        # the clipped gradients go to the optimizer's own buffers: the others stay what they were
        if c["flat"]:
            flat = {k: normal(sum(n for n, t in zip(sizes, kinds) if t is k), std=std, dtype=k) for k in dict.fromkeys(kinds)}
            s["buffers"] = {k: torch.empty_like(t) for k, t in flat.items()}
            s["grads"], s["out"] = _views(flat, c, kinds), _views(s["buffers"], c, kinds)
        else:
            s["grads"] = [normal(*sh, std=std, dtype=k) for sh, k in zip(_shapes(c), kinds)]
            s["out"] = [torch.empty_like(t) for t in s["grads"]]
    return s


# ---------------------------------------------------------------------------------------------- passes

def _values(codes, scale):
    """Rows in E4M3 with 1x128 scales, as fp32."""
    v = codes.view(E4M3).float()
    return (v.view(v.shape[0], -1, BLK) * _scale_in(scale)[..., None]).view(v.shape)


def _weight_values(codes, scale):
    return codes.view(E4M3).float() * _scale_in(scale).repeat_interleave(BLK, -2).repeat_interleave(BLK, -1)


def _coded(q, e):
    return {"values": q.view(E4M3), "scale": e.view(E8M0)}


def _product(s):
    """Each group's rows times its weight, in a batch of groups padded to the largest."""
    x, W, off = _values(s["X"], s["X_scale"]), _weight_values(s["W"], s["W_scale"]), s["offsets"].long()
    R = x.shape[0]
    row = torch.arange(R, device=off.device)
    e = torch.bucketize(row, off[1:], right=True)
    at = off[:-1, None] + torch.arange(max(1, s["most"]), device=off.device)
    y = torch.matmul(x[at.clamp_max(max(R - 1, 0))], W if s["backward"] else W.transpose(1, 2))
    return y[e, row - off[e]]


def _plain_swiglu(s):
    i = s["I"]
    if not s["backward"]:
        gu = _product(s)
        g, u = gu[:, :i], gu[:, i:]
        out = {"A": _coded(*_quant_rows(g / (1 + torch.exp(-g)) * u, "ue8m0"))}
        if s["keep"]:
            out["kept"] = _coded(*_quant_rows(gu, "ue8m0"))
        return out
    da, gu = _product(s), _values(s["GU"], s["GU_scale"])
    g, u = gu[:, :i], gu[:, i:]
    sig = 1 / (1 + torch.exp(-g))
    d = torch.cat([da * u * sig * (1 + g * (1 - sig)), da * g * sig], 1)
    return {"dGU": d.to(torch.bfloat16), "coded": _coded(*_quant_rows(d, "ue8m0"))}


def _plain_rms_norm(s):
    w = s["w"].float()
    if not s["backward"]:
        t = s["X"] if s["res"] is None else (s["X"].float() + s["res"].float()).to(torch.bfloat16)
        v = t.float()
        rstd = torch.rsqrt((v * v).mean(1) + EPS)
        y = v * rstd[:, None] * w
        out = {"Y": y.to(torch.bfloat16), "rstd": rstd}
        if s["res"] is not None:
            out["S"] = t
        if s["fp8"]:
            out["coded"] = _coded(*_quant_rows(y, "ue8m0"))
        return out
    dy, r = s["dY"].float(), s["rstd"][:, None]
    xh = s["S"].float() * r
    d = dy * w
    dx = r * (d - xh * (d * xh).mean(1, keepdim=True))
    if s["dS"] is not None:
        dx = dx + s["dS"].float()
    dw = (dy * xh).sum(0)
    return {"dX": dx.to(torch.bfloat16), "dw": dw if s["add"] is None else s["add"] + dw}


def _plain_clip(s):
    # (sums of up to some 10^8 squares)
    norm = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum().sqrt().float().view(1)
    if not s["clip"]:
        return {"norm": norm}
    c = (s["max_norm"] / (norm + 1e-6)).clamp_max(1)
    return {"norm": norm, "grads": _joined(s, [(t.float() * c).to(t.dtype) for t in s["grads"]])}


def run(s):
    if not own:
        return {"rms_norm": _plain_rms_norm, "swiglu": _plain_swiglu, "clip": _plain_clip}[s["op"]](s)
    import combine_moe_route_02_gb300 as moe
    if s["op"] == "rms_norm":
        if s["backward"]:
            r = moe.rms_norm_backward(s["dY"], s["S"], s["w"], s["rstd"], dS=s["dS"], add=s["add"])
            return {"dX": r.dX, "dw": r.dweight}
        r = moe.rms_norm(s["X"], s["w"], residual=s["res"], eps=EPS, fp8=s["fp8"], scale_format="ue8m0")
        out = {"Y": r.Y, "rstd": r.rstd}
        if s["res"] is not None:
            out["S"] = r.S
        if s["fp8"]:
            out["coded"] = _coded(r.Y_fp8, r.Y_scale)
        return out
    if s["op"] == "swiglu":
        if s["backward"]:
            r = moe.expert_swiglu_backward(s["X"], s["X_scale"], s["W"], s["W_scale"], s["GU"], s["GU_scale"], s["offsets"], scale_format="ue8m0")
            return {"dGU": r.dGU, "coded": _coded(r.dGU_fp8, r.dGU_scale)}
        r = moe.expert_swiglu(s["X"], s["X_scale"], s["W"], s["W_scale"], s["offsets"], keep=s["keep"], scale_format="ue8m0")
        out = {"A": _coded(r.A_fp8, r.A_scale)}
        if s["keep"]:
            out["kept"] = _coded(r.GU_fp8, r.GU_scale)
        return out
    if not s["clip"]:
        return {"norm": moe.grad_norm(s["grads"])}
    norm = moe.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])
    return {"norm": norm, "grads": list(s["buffers"].values()) if s["flat"] else s["out"]}


# ---------------------------------------------------------------------------------------------- in 64 bits

def _table():
    """The value of each E4M3 code."""
    code = np.arange(256)
    sign, e, m = np.where(code & 128, -1.0, 1.0), (code >> 3) & 15, code & 7
    v = sign * np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(code & 127) == 127] = np.nan
    return torch.from_numpy(v).to(DEV)


def _two_to(n):
    """2^n in 64 bits for whole n, by its bits."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _real(codes, scale, rows):
    """E4M3 with a scale for each rows x 128 block, in 64 bits."""
    v = _table()[codes.long()]
    sc = _two_to(scale.long() - 127) if scale.dtype == torch.uint8 else scale.double()
    i = torch.arange(v.shape[-2], device=DEV) // rows
    j = torch.arange(v.shape[-1], device=DEV) // BLK
    return v * sc[..., i, :][..., j]


def _round_e4m3(v):
    """The nearest E4M3 value, ties to the even one, kept within 448."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -40))).clamp_min(-6)
    step = _two_to(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_rows(x):
    """E4M3 values and the scales of 1x128 blocks."""
    b = x.unflatten(1, (-1, BLK))
    # the scale is defined by a product in 32 bits
    t = (b.abs().amax(-1).clamp_min(1e-4).float() * torch.tensor(RCP448, device=DEV)).double()
    s = _two_to(torch.round(torch.log2(t)))
    s = torch.where(s < t, 2 * s, s)
    s = torch.where(s / 2 >= t, s / 2, s)
    return _round_e4m3(b / s[..., None]).flatten(1), s


def _exact_swiglu(c, s):
    i, off, parts = c["I"], s["offsets"].tolist(), []
    for e in range(c["E"]):
        a, b = off[e], off[e + 1]
        x, W = _real(s["X"][a:b], s["X_scale"][a:b], 1), _real(s["W"][e], s["W_scale"][e], BLK)
        if c["backward"]:
            gu, da = _real(s["GU"][a:b], s["GU_scale"][a:b], 1), x @ W
            g, u = gu[:, :i], gu[:, i:]
            sig = torch.sigmoid(g)
            d = torch.cat((da * u * (sig + g * sig * torch.sigmoid(-g)), da * g * sig), 1)
            parts.append((d,) + _exact_rows(d))
        else:
            gu = x @ W.T
            part = _exact_rows(gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:])
            parts.append(part + _exact_rows(gu) if c["keep"] else part)
    p = [torch.cat(t) for t in zip(*parts)]
    if c["backward"]:
        return {"dGU": p[0], "coded": {"values": p[1], "scale": p[2]}}
    out = {"A": {"values": p[0], "scale": p[1]}}
    if c["keep"]:
        out["kept"] = {"values": p[2], "scale": p[3]}
    return out


def _exact_rms_norm(c, s):
    w, parts, dw = s["w"].double(), [], torch.zeros(c["H"], dtype=torch.float64, device=DEV)
    for r in range(0, c["N"], 8192):
        at = slice(r, r + 8192)
        if c["backward"]:
            v, dy, rstd = s["S"][at].double(), s["dY"][at].double(), s["rstd"][at].double()[:, None]
            dw += torch.einsum("nh,nh,n->h", dy, v, rstd[:, 0])
            d = dy * w * rstd
            d -= v * rstd ** 3 * torch.einsum("nh,nh->n", dy * w, v)[:, None] / c["H"]
            parts.append((d if s["dS"] is None else d + s["dS"][at].double(),))
        else:
            t = s["X"][at].double()
            if s["res"] is not None:
                t = t + s["res"][at].double()
            # what is normed is the stream as it is kept, in bf16
            v = t.to(torch.bfloat16).double()
            rstd = (torch.linalg.vector_norm(v, dim=1).square() / c["H"] + EPS).pow(-0.5)
            y = v * w * rstd[:, None]
            parts.append((y, rstd, t) + (_exact_rows(y) if c["fp8"] else ()))
    p = [torch.cat(t) for t in zip(*parts)]
    if c["backward"]:
        return {"dX": p[0], "dw": dw if s["add"] is None else dw + s["add"].double()}
    out = {"Y": p[0], "rstd": p[1]}
    if s["res"] is not None:
        out["S"] = p[2]
    if c["fp8"]:
        out["coded"] = {"values": p[3], "scale": p[4]}
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rms_norm":
        return _exact_rms_norm(c, s)
    if c["op"] == "swiglu":
        return _exact_swiglu(c, s)
    norm = torch.stack([torch.linalg.vector_norm(t.double()) for t in s["grads"]]).norm().view(1)
    if not c["clip"]:
        return {"norm": norm}
    by = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    return {"norm": norm, "grads": _joined(s, [t.double() * by for t in s["grads"]])}
