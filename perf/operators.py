"""The operators of the mixture-of-experts layer behind the router: what a pass of each computes and costs.

  gemm      the experts' matrix products in E4M3 with power-of-two scales of 1x128 (rows) and 128x128 (weights)
            blocks, over ragged groups of rows; `transpose` is the input gradient's product
  wgrad     the weight gradient of those products, read from the rows' E4M3 checkpoint
  swiglu    the gated activation between the two products: E4M3 out, its input kept in E4M3; `backward` its gradient
  quantize  E4M3 weights with 128x128 scales from bf16 ones
  layer     the whole layer (router, both products, combine) for a few tokens

`run` computes them in plain torch operations where `own` is false and through the package where it is true; `exact`
computes them in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLK = 128
E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
RCP448 = float(np.float32(1) / np.float32(448))


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # 65 tokens of a small layer: several experts hold one row or none, the call is its own latency
        dict(name="gemm_65tok_e16", op="gemm", N=65, E=16, K=2, rows=512, cols=256, transpose=False, skew=0.0, fmt="fp32"),
        # the up/gate product of a training step of 16384 tokens, 128 experts, top 8
        dict(name="gemm_up_16384tok_e128", op="gemm", N=16384, E=128, K=8, rows=2048, cols=2048, transpose=False, skew=0.0, fmt="ue8m0"),
        # input gradient under an uneven load, 64 experts, top 2, an odd number of tokens
        dict(name="gemm_dx_skewed_e64", op="gemm", N=16381, E=64, K=2, rows=1024, cols=4096, transpose=True, skew=0.5, fmt="fp32"),
        # weight gradient of a small step added to a 32-bit buffer, some experts without rows
        dict(name="wgrad_1023tok_e64_add", op="wgrad", N=1023, E=64, K=2, rows=512, cols=1024, skew=1.0, fmt="fp32", add=True),
        # weight gradient of the up/gate product of the 16384-token step, in bf16
        dict(name="wgrad_up_16384tok_e128", op="wgrad", N=16384, E=128, K=8, rows=2048, cols=2048, skew=0.0, fmt="ue8m0", add=False),
        # activation of the 16384-token step, forward with its checkpoint
        dict(name="swiglu_131072x1024", op="swiglu", R=131072, I=1024, backward=False, fmt="ue8m0"),
        # gradient of the activation, an odd number of rows
        dict(name="swiglu_bwd_32761x1024", op="swiglu", R=32761, I=1024, backward=True, fmt="fp32"),
        # one expert matrix, and the up/gate matrices of a layer of 64 experts after an optimizer step
        dict(name="quantize_1x512x256", op="quantize", E=1, rows=512, cols=256, fmt="ue8m0"),
        dict(name="quantize_64x2048x2048", op="quantize", E=64, rows=2048, cols=2048, fmt="fp32"),
        # decoding: one sequence, an odd small batch, and the most tokens a call takes
        dict(name="layer_1tok_e128", op="layer", N=1, H=2048, I=1024, E=128, K=8, fmt="ue8m0", residual=True),
        dict(name="layer_13tok_e64", op="layer", N=13, H=2048, I=512, E=64, K=4, fmt="fp32", residual=False),
        dict(name="layer_64tok_e128", op="layer", N=64, H=2048, I=1024, E=128, K=8, fmt="ue8m0", residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dim(rng, lo, hi, step):
    while True:
        v = max(lo, _log(rng, lo, hi) // step * step)
        if v not in (1536, 3072):
            return v


def draw(rng):
    while True:
        op = rng.choice(["gemm", "gemm", "wgrad", "swiglu", "quantize", "layer"])
        fmt = rng.choice(["fp32", "ue8m0"])
        if op in ("gemm", "wgrad"):
            E = rng.choice([1, 5, 16, 64, 128])
            K = min(E, rng.choice([1, 2, 4, 8]))
            c = dict(op=op, N=_log(rng, 1, 16384), E=E, K=K, skew=rng.choice([0.0, 0.5, 1.0]), fmt=fmt)
            if op == "gemm":
                c["transpose"] = rng.random() < 0.5
                # the reduction is whole in blocks of 128, the other side need not be
                c["rows"] = _dim(rng, 128, 2048, 128 if c["transpose"] else 16)
                c["cols"] = _dim(rng, 128, 4096, 16 if c["transpose"] else 128)
            else:
                c.update(rows=_dim(rng, 128, 2048, 8), cols=_dim(rng, 128, 4096, 128), add=rng.random() < 0.5)
            # the plain form pads every group to the largest
            if c["N"] * K * c["rows"] * c["cols"] > 131072 * 2048 * 2048 or (c["skew"] and c["N"] * K > 32768):
                continue
        elif op == "swiglu":
            c = dict(op=op, R=_log(rng, 1, 131072), I=_dim(rng, 128, 2048, 128), backward=rng.random() < 0.5, fmt=fmt)
            if c["R"] * c["I"] > 131072 * 1024:
                continue
        elif op == "quantize":
            c = dict(op=op, E=rng.choice([1, 5, 16, 64]), rows=_dim(rng, 128, 2048, 8), cols=_dim(rng, 128, 2048, 8), fmt=fmt)
        else:
            E = rng.choice([8, 16, 64, 128])
            c = dict(op=op, N=_log(rng, 1, 64), H=_dim(rng, 256, 2048, 128), I=_dim(rng, 128, 1024, 128), E=E,
                     K=min(E, rng.choice([1, 2, 4, 8])), fmt=fmt, residual=rng.random() < 0.5)
        if 3072 not in (c.get("N"), c.get("R"), c.get("N", 0) * c.get("K", 0)):
            return c


def _touched(c):
    """Experts that N tokens of K distinct experts reach, on average."""
    return c["E"] * (1 - (1 - c["K"] / c["E"]) ** c["N"])


def work(c):
    sb = 1 if c["fmt"] == "ue8m0" else 4
    if c["op"] in ("gemm", "wgrad"):
        R, n, k = c["N"] * c["K"], c["rows"], c["cols"]
        flops = 2 * R * n * k
        if c["op"] == "gemm":
            red, out = (n, k) if c["transpose"] else (k, n)
            weights = _touched(c) * (n * k + sb * -(-n // BLK) * -(-k // BLK))
            return {"bytes": R * (red + sb * red // BLK + 2 * out) + weights + 4 * (c["E"] + 1), "flops": flops}
        moved = c["E"] * n * k * (8 if c["add"] else 2)   # experts without rows are written too
        return {"bytes": R * (2 * n + k + sb * k // BLK) + moved + 4 * (c["E"] + 1), "flops": flops}
    if c["op"] == "swiglu":
        R, i = c["R"], c["I"]
        if c["backward"]:   # dA, the checkpoint of both halves; dGU in bf16 and E4M3
            return {"bytes": R * (2 * i + 2 * (i + sb * i // BLK) + 4 * i + 2 * (i + i // BLK)), "flops": 20 * R * i}
        return {"bytes": R * (4 * i + 3 * (i + sb * i // BLK)), "flops": 10 * R * i}
    if c["op"] == "quantize":
        n = c["E"] * c["rows"] * c["cols"]
        return {"bytes": 3 * n + sb * c["E"] * -(-c["rows"] // BLK) * -(-c["cols"] // BLK), "flops": 2 * n}
    N, H, i, E, K = c["N"], c["H"], c["I"], c["E"], c["K"]
    per = 3 * H * i + sb * 3 * (H // BLK) * (i // BLK)
    return {"bytes": H * E * 2 + _touched(c) * per + N * H * (6 if c["residual"] else 4) + N * K * 8,
            "flops": 2 * N * H * E + 6 * N * K * H * i}


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) + 1000003)


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
    """[E, n, k] -> E4M3 codes (uint8) and scales of 128x128 blocks, the last ones cut at the edges."""
    E, n, k = W.shape
    nb, kb = -(-n // BLK), -(-k // BLK)
    a = torch.nn.functional.pad(W.abs(), (0, kb * BLK - k, 0, nb * BLK - n)).view(E, nb, BLK, kb, BLK)
    s, e = _pow2ceil(a.amax((2, 4)).float().clamp_min(1e-4) * RCP448)
    q = torch.empty((E, n, k), dtype=torch.uint8, device=W.device)
    per = s.repeat_interleave(BLK, 1)[:, :n].repeat_interleave(BLK, 2)[:, :, :k]
    q.copy_((W.float() / per).to(E4M3).view(torch.uint8))
    return q, _scale_out(s, e, fmt)


def _offsets(c, g):
    """Rows of each expert: every token takes K different experts, by a preference when the load is skewed."""
    pref = torch.rand((c["N"], c["E"]), generator=g, device=DEV).log().neg().log().neg()
    pref -= c["skew"] * torch.arange(1, c["E"] + 1, device=DEV).log()
    idx = pref.topk(c["K"], dim=1).indices
    off = torch.zeros(c["E"] + 1, dtype=torch.int32, device=DEV)
    off[1:] = torch.bincount(idx.flatten(), minlength=c["E"]).cumsum(0)
    return off


def prepare(c, seed):
    g = _gen(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)

    s = dict(c)
    if c["op"] in ("gemm", "wgrad"):
        s["offsets"] = _offsets(c, g)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        R, n, k = c["N"] * c["K"], c["rows"], c["cols"]
        x = normal(R, n if c.get("transpose") else k)
        s["X"], s["X_scale"] = _quant_rows(x.float(), c["fmt"])
        if c["op"] == "gemm":
            s["W"], s["W_scale"] = _quant_weight(normal(c["E"], n, k, std=k ** -0.5), c["fmt"])
        else:
            s["dY"] = normal(R, n)
            if c["add"]:
                s["dW"] = torch.randn((c["E"], n, k), generator=g, device=DEV)
    elif c["op"] == "swiglu":
        if c["backward"]:
            s["dA"] = normal(c["R"], c["I"])
            s["GU"], s["GU_scale"] = _quant_rows(normal(c["R"], 2 * c["I"]).float(), c["fmt"])
        else:
            s["GU"] = normal(c["R"], 2 * c["I"])
    elif c["op"] == "quantize":
        s["W"] = normal(c["E"], c["rows"], c["cols"], std=c["cols"] ** -0.5)
    else:
        N, H, i, E = c["N"], c["H"], c["I"], c["E"]
        s["X"], s["W_gate"] = normal(N, H), normal(H, E, std=H ** -0.5)
        s["W1"], s["W1_scale"] = _quant_weight(normal(E, 2 * i, H, std=H ** -0.5), c["fmt"])
        s["W2"], s["W2_scale"] = _quant_weight(normal(E, H, i, std=i ** -0.5), c["fmt"])
        s["res"] = normal(N, H) if c["residual"] else None
    return s


# ---------------------------------------------------------------------------------------------- passes

def _values(codes, scale):
    """Rows in E4M3 with 1x128 scales, as fp32."""
    v = codes.view(E4M3).float()
    return (v.view(v.shape[0], -1, BLK) * _scale_in(scale)[..., None]).view(v.shape)


def _weight_values(codes, scale):
    n, k = codes.shape[-2:]
    per = _scale_in(scale).repeat_interleave(BLK, -2)[..., :n, :].repeat_interleave(BLK, -1)[..., :k]
    return codes.view(E4M3).float() * per


def _groups(s, R):
    """Where row r lies in a batch of groups padded to the largest: its group, its place, and each place's row."""
    off = s["offsets"].long()
    row = torch.arange(R, device=off.device)
    e = torch.bucketize(row, off[1:], right=True)
    at = off[:-1, None] + torch.arange(max(1, s["most"]), device=off.device)
    return e, row - off[e], at.clamp_max(max(R - 1, 0)), at < off[1:, None]


def _plain_gemm(s):
    x = _values(s["X"], s["X_scale"])
    W = _weight_values(s["W"], s["W_scale"])
    e, place, at, _ = _groups(s, x.shape[0])
    y = torch.matmul(x[at], W if s["transpose"] else W.transpose(1, 2))
    return y[e, place].to(torch.bfloat16)


def _plain_wgrad(s):
    x = _values(s["X"], s["X_scale"])
    _, _, at, there = _groups(s, x.shape[0])
    d = s["dY"].float()[at] * there[..., None]
    dW = torch.matmul(d.transpose(1, 2), x[at])
    return s["dW"] + dW if s["add"] else dW.to(torch.bfloat16)


def _coded(q, e):
    return {"values": q.view(E4M3), "scale": e.view(E8M0)}


def _plain_swiglu(s):
    i = s["I"]
    if not s["backward"]:
        gu = s["GU"].float()
        g, u = gu[:, :i], gu[:, i:]
        return {"A": _coded(*_quant_rows(g / (1 + torch.exp(-g)) * u, "ue8m0")),
                "kept": _coded(*_quant_rows(gu, "ue8m0"))}
    gu, da = _values(s["GU"], s["GU_scale"]), s["dA"].float()
    g, u = gu[:, :i], gu[:, i:]
    sig = 1 / (1 + torch.exp(-g))
    d = torch.cat([da * u * sig * (1 + g * (1 - sig)), da * g * sig], 1)
    return {"dGU": d.to(torch.bfloat16), "coded": _coded(*_quant_rows(d, "ue8m0"))}


def _plain_layer(s):
    N, H, i, K = s["N"], s["H"], s["I"], s["K"]
    x = s["X"].float()
    top, idx = torch.matmul(x, s["W_gate"].float()).sort(dim=1, descending=True, stable=True)
    idx = idx[:, :K]
    w = torch.exp(top[:, :K] - top[:, :1])
    w = w / w.sum(1, keepdim=True)
    e = idx.reshape(-1)
    xq = _values(*_quant_rows(x, "fp32")).repeat_interleave(K, 0)
    gu = torch.matmul(_weight_values(s["W1"][e], s["W1_scale"][e]), xq[..., None])[..., 0]
    g, u = gu[:, :i], gu[:, i:]
    a = _values(*_quant_rows(g / (1 + torch.exp(-g)) * u, "fp32"))
    y = torch.matmul(_weight_values(s["W2"][e], s["W2_scale"][e]), a[..., None]).view(N, K, H)
    out = (y * w[..., None]).sum(1)
    if s["res"] is not None:
        out = out + s["res"].float()
    return {"out": out.to(torch.bfloat16), "idx": idx.to(torch.int32), "w": w}


def run(s):
    if not own:
        if s["op"] == "quantize":
            q, scale = _quant_weight(s["W"], s["fmt"])
            return {"values": q.view(E4M3), "scale": scale.view(E8M0) if s["fmt"] == "ue8m0" else scale}
        return {"gemm": _plain_gemm, "wgrad": _plain_wgrad, "swiglu": _plain_swiglu, "layer": _plain_layer}[s["op"]](s)
    import combine_moe_route_02_gb300 as moe
    if s["op"] == "gemm":
        return moe.expert_gemm(s["X"], s["X_scale"], s["W"], s["W_scale"], s["offsets"], transpose=s["transpose"])
    if s["op"] == "wgrad":
        if s["add"]:
            # the sum goes to a buffer of its own, so that a pass can be repeated on the same state
            return moe.expert_wgrad(s["dY"], s["X"], s["X_scale"], s["offsets"], add=s["dW"])
        return moe.expert_wgrad(s["dY"], s["X"], s["X_scale"], s["offsets"], dtype=torch.bfloat16)
    if s["op"] == "swiglu":
        if s["backward"]:
            r = moe.swiglu_backward(s["dA"], s["GU"], s["GU_scale"], scale_format="ue8m0")
            return {"dGU": r.dGU, "coded": _coded(r.dGU_fp8, r.dGU_scale)}
        r = moe.swiglu(s["GU"], scale_format="ue8m0")
        return {"A": _coded(r.A_fp8, r.A_scale), "kept": _coded(r.GU_fp8, r.GU_scale)}
    if s["op"] == "quantize":
        q, scale = moe.quantize_weight(s["W"], scale_format=s["fmt"])
        return {"values": q.view(E4M3), "scale": scale.view(E8M0) if s["fmt"] == "ue8m0" else scale}
    r = moe.moe_layer(s["X"], s["W_gate"], s["K"], s["W1"], s["W1_scale"], s["W2"], s["W2_scale"], residual=s["res"])
    return {"out": r.out, "idx": r.topk_idx, "w": r.topk_w}


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


def _real_scale(scale):
    return _two_to(scale.long() - 127) if scale.dtype == torch.uint8 else scale.double()


def _real(codes, scale, rows, cols):
    """E4M3 with a scale for each rows x cols block, in 64 bits."""
    v = _table()[codes.long()]
    sc = _real_scale(scale)
    i = torch.arange(v.shape[-2], device=DEV) // rows
    j = torch.arange(v.shape[-1], device=DEV) // cols
    return v * sc[..., i, :][..., j]


def _round_e4m3(v):
    """The nearest E4M3 value, ties to the even one, kept within 448."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -40))).clamp_min(-6)
    step = _two_to(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _block_scale(amax):
    # the scale is defined by a product in 32 bits
    t = (amax.clamp_min(1e-4).float() * torch.tensor(RCP448, device=DEV)).double()
    s = _two_to(torch.round(torch.log2(t)))
    s = torch.where(s < t, 2 * s, s)
    return torch.where(s / 2 >= t, s / 2, s)


def _exact_rows(x):
    b = x.unflatten(1, (-1, BLK))
    s = _block_scale(b.abs().amax(-1))
    return _round_e4m3(b / s[..., None]).flatten(1), s


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op in ("gemm", "wgrad"):
        off = s["offsets"].tolist()
        pieces = []
        for e in range(c["E"]):
            a, b = off[e], off[e + 1]
            x = _real(s["X"][a:b], s["X_scale"][a:b], 1, BLK)
            if op == "gemm":
                W = _real(s["W"][e], s["W_scale"][e], BLK, BLK)
                pieces.append(x @ (W if c["transpose"] else W.T))
            else:
                d = s["dY"][a:b].double().T @ x
                # the sample that is compared does not need 64 bits kept where the output is bf16
                pieces.append(d + s["dW"][e] if c["add"] else d)
        return torch.cat(pieces) if op == "gemm" else torch.stack(pieces)
    if op == "swiglu":
        i, parts = c["I"], []
        for r in range(0, c["R"], 16384):
            if c["backward"]:
                gu, da = _real(s["GU"][r:r + 16384], s["GU_scale"][r:r + 16384], 1, BLK), s["dA"][r:r + 16384].double()
                g, u = gu[:, :i], gu[:, i:]
                sig = torch.sigmoid(g)
                d = torch.cat((da * u * (sig + g * sig * torch.sigmoid(-g)), da * g * sig), 1)
                q, sc = _exact_rows(d)
                parts.append((d, q, sc))
            else:
                gu = s["GU"][r:r + 16384].double()
                q, sc = _exact_rows(gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:])
                parts.append((q, sc) + _exact_rows(gu))
        p = [torch.cat(t) for t in zip(*parts)]
        if c["backward"]:
            return {"dGU": p[0], "coded": {"values": p[1], "scale": p[2]}}
        return {"A": {"values": p[0], "scale": p[1]}, "kept": {"values": p[2], "scale": p[3]}}
    if op == "quantize":
        n, k = c["rows"], c["cols"]
        nb, kb = -(-n // BLK), -(-k // BLK)
        scale = torch.empty((c["E"], nb, kb), dtype=torch.float64, device=DEV)
        values = torch.empty((c["E"], n, k), dtype=torch.float64, device=DEV)
        for i in range(nb):
            for j in range(kb):
                at = (slice(None), slice(i * BLK, (i + 1) * BLK), slice(j * BLK, (j + 1) * BLK))
                w = s["W"][at].double()
                scale[:, i, j] = _block_scale(w.abs().amax((1, 2)))
                values[at] = _round_e4m3(w / scale[:, i, j, None, None])
        return {"values": values, "scale": scale}
    N, H, i, K = c["N"], c["H"], c["I"], c["K"]
    x = s["X"].double()
    logits = x @ s["W_gate"].double()
    q, sc = _exact_rows(x)
    xq = (q.unflatten(1, (-1, BLK)) * sc[..., None]).flatten(1)
    out = torch.zeros((N, H), dtype=torch.float64, device=DEV) if s["res"] is None else s["res"].double()
    idx = torch.empty((N, K), dtype=torch.int32, device=DEV)
    w = torch.empty((N, K), dtype=torch.float64, device=DEV)
    for n in range(N):
        order = sorted(range(c["E"]), key=lambda e, row=logits[n].tolist(): (-row[e], e))[:K]
        w[n] = torch.softmax(logits[n][order], 0)
        idx[n] = torch.tensor(order, dtype=torch.int32, device=DEV)
        for k, e in enumerate(order):
            gu = _real(s["W1"][e], s["W1_scale"][e], BLK, BLK) @ xq[n]
            q, sc = _exact_rows((gu[:i] * torch.sigmoid(gu[:i]) * gu[i:])[None])
            a = (q.unflatten(1, (-1, BLK)) * sc[..., None]).flatten(1)[0]
            out[n] += w[n, k] * (_real(s["W2"][e], s["W2_scale"][e], BLK, BLK) @ a)
    return {"out": out, "idx": idx, "w": w}
