"""A pre-norm mixture-of-experts block, trained for a few steps with the package's kernels.

    s   = x + attn                    the residual stream               rms_norm (one pass: s, y, y in E4M3)
    y   = rms(s) * w
    out = s + sum_k p_k expert_k(y) + shared(y)

Routing, dispatch and combine as in examples/moe_mlp.py; both products of an expert's gate and up halves run with the
activation behind them (expert_swiglu), also for the shared expert, which reads the norm's E4M3 rows as they are.  The
backward pass goes down to the gradients of x and w; the step is plain gradient descent with the norm of all gradients
clipped on the device.  (The router's own weights are left as they are.)

    python examples/moe_block.py [--tokens 4096 --hidden 1024 --inner 512 --experts 64 --topk 4 --steps 8]
"""
import argparse
import os
import sys
from types import SimpleNamespace

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import combine_moe_route_02_gb300 as moe

FMT = "ue8m0"


def quantized(W):
    return moe.quantize_weight(W.to(torch.bfloat16), scale_format=FMT)


def rows_in_e4m3(t):
    """bf16 rows as E4M3 codes and 1x128 scales."""
    ident = torch.arange(t.shape[0], dtype=torch.int32, device=t.device)
    return moe.permute(t, ident, K=1, fp8=True, bf16=False, scale_format=FMT)[1:3]


def forward(x, attn, w, W_gate, K, W1q, W2q, V1q, V2q):
    """The block's output, and what its backward pass needs.  W1q, W2q: the experts; V1q, V2q: the shared one."""
    n = moe.rms_norm(attn, w, residual=x, fp8=True, scale_format=FMT)
    idx, p = moe.route(n.Y, W_gate, K)
    d = moe.dispatch(idx, W_gate.shape[1], n.Y, fp8=True, bf16=False, scale_format=FMT)
    h = moe.expert_swiglu(d.X_fp8, d.X_scale, *W1q, d.expert_offsets, scale_format=FMT)
    e = moe.expert_gemm(h.A_fp8, h.A_scale, *W2q, d.expert_offsets)
    hs = moe.expert_swiglu(n.Y_fp8, n.Y_scale, *V1q, scale_format=FMT)
    out = moe.combine(e, d.row_map, p, residual=n.S) + moe.expert_gemm(hs.A_fp8, hs.A_scale, *V2q)
    return out, SimpleNamespace(n=n, p=p, d=d, h=h, hs=hs)


def backward(dout, saved, w, W1q, W2q, V1q, V2q):
    """Gradients of W1, W2, V1, V2 and w, and of x (and attn alike)."""
    n, p, d, h, hs = saved.n, saved.p, saved.d, saved.h, saved.hs
    K, off, slot = p.shape[1], d.expert_offsets, d.src_slot.long()
    # the combine's gradient: row r of slot s = n K + k gets p[n, k] dout[n]
    dE = (dout[slot // K].float() * p.flatten()[slot, None]).to(torch.bfloat16)
    g = moe.expert_swiglu_backward(*rows_in_e4m3(dE), *W2q, h.GU_fp8, h.GU_scale, off, scale_format=FMT)
    dW2 = moe.expert_wgrad(dE, h.A_fp8, h.A_scale, off)
    dW1 = moe.expert_wgrad(g.dGU, d.X_fp8, d.X_scale, off)
    dY = moe.combine(moe.expert_gemm(g.dGU_fp8, g.dGU_scale, *W1q, off, transpose=True), d.row_map, torch.ones_like(p))
    g = moe.expert_swiglu_backward(*rows_in_e4m3(dout), *V2q, hs.GU_fp8, hs.GU_scale, scale_format=FMT)
    dV2 = moe.expert_wgrad(dout, hs.A_fp8, hs.A_scale)[0]
    dV1 = moe.expert_wgrad(g.dGU, n.Y_fp8, n.Y_scale)[0]
    dY = dY + moe.expert_gemm(g.dGU_fp8, g.dGU_scale, *V1q, transpose=True)
    r = moe.rms_norm_backward(dY, n.S, w, n.rstd, dS=dout)
    return [dW1, dW2, dV1, dV2, r.dweight], r.dX


def main(argv=None):
    a = argparse.ArgumentParser(description=__doc__.split("\n", 1)[0])
    for name, default in (("tokens", 4096), ("hidden", 1024), ("inner", 512), ("experts", 64), ("topk", 4), ("steps", 8)):
        a.add_argument("--" + name, type=int, default=default)
    a.add_argument("--rate", type=float, default=1.0)
    a.add_argument("--max-norm", type=float, default=1.0)
    a = a.parse_args(argv)
    moe.build()
    dev, H, I, E, K = torch.device("cuda"), a.hidden, a.inner, a.experts, a.topk
    gen = torch.Generator().manual_seed(0)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen) * std).to(dev)

    W_gate = normal(H, E, std=H ** -0.5).to(torch.bfloat16)
    params = [normal(E, 2 * I, H, std=H ** -0.5), normal(E, H, I, std=I ** -0.5),
              normal(2 * I, H, std=H ** -0.5), normal(H, I, std=I ** -0.5), torch.ones(H, device=dev)]
    x, attn, target = (normal(a.tokens, H).to(torch.bfloat16) for _ in range(3))
    norms = []
    for step in range(a.steps):
        coded = [quantized(W) for W in params[:4]]
        out, saved = forward(x, attn, params[4], W_gate, K, *coded)
        diff = out.float() - target.float()
        grads, dx = backward((diff * (1 / a.tokens)).to(torch.bfloat16), saved, params[4], *coded)
        norm = moe.clip_grad_norm(grads, a.max_norm)         # the host does not wait for it
        for W, dW in zip(params, grads):
            W -= a.rate * dW
        norms.append(float(norm))
        print(f"step {step}: loss {float(diff.square().mean()):.5f}, gradient norm {norms[-1]:.5f}, |dx| {float(dx.float().norm()):.5f}")
    return norms, [float(moe.grad_norm(grads))]


if __name__ == "__main__":
    main()
