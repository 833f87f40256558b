"""A mixture-of-experts layer trained and then served with the package's kernels.

The layer (router, gated MLP of the top-K experts, weighted sum) learns to imitate another
one with random weights: a few steps of gradient descent on the experts' weights, with
everything between router and combine in E4M3, forward and backward, and nothing but E4M3
kept in between.  Then a few tokens go through the whole layer in one launch.

    python examples/moe_mlp.py [--tokens 4096 --hidden 1024 --inner 512 --experts 64 --topk 4 --steps 8]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import combine_moe_route_02_gb300 as moe


def quantized(W):
    return moe.quantize_weight(W.to(torch.bfloat16), scale_format="ue8m0")


def forward(X, W_gate, K, W1q, W2q):
    """Output, and what the backward pass needs."""
    E = W_gate.shape[1]
    idx, w = moe.route(X, W_gate, K)
    d = moe.dispatch(idx, E, X, fp8=True, bf16=False, scale_format="ue8m0")
    gu = moe.expert_gemm(d.X_fp8, d.X_scale, *W1q, d.expert_offsets)
    h = moe.swiglu(gu, scale_format="ue8m0")
    y = moe.expert_gemm(h.A_fp8, h.A_scale, *W2q, d.expert_offsets)
    return moe.combine(y, d.row_map, w), (d, h, w)


def backward(dout, saved, W1q, W2q, dW1=None, dW2=None):
    """Gradients of the weights (added to dW1, dW2 where given) and of the layer's input through the experts."""
    d, h, w = saved
    K = w.shape[1]
    off = d.expert_offsets
    # the combine's gradient: row r of slot s = n K + k gets w[n, k] dout[n]
    slot = d.src_slot.long()
    dY = (dout[slot // K].float() * w.flatten()[slot, None]).to(torch.bfloat16)
    rows = torch.arange(dY.shape[0], dtype=torch.int32, device=dY.device)
    dY8, dY8s = moe.permute(dY, rows, K=1, fp8=True, bf16=False, scale_format="ue8m0")[1:3]
    dA = moe.expert_gemm(dY8, dY8s, *W2q, off, transpose=True)
    g = moe.swiglu_backward(dA, h.GU_fp8, h.GU_scale, scale_format="ue8m0")
    dW2 = moe.expert_wgrad(dY, h.A_fp8, h.A_scale, off, add=dW2, out=dW2)
    dW1 = moe.expert_wgrad(g.dGU, d.X_fp8, d.X_scale, off, add=dW1, out=dW1)
    dXr = moe.expert_gemm(g.dGU_fp8, g.dGU_scale, *W1q, off, transpose=True)
    dX = moe.combine(dXr, d.row_map, torch.ones_like(w))
    return dW1, dW2, dX


def main(argv=None):
    a = argparse.ArgumentParser(description=__doc__.split("\n", 1)[0])
    for name, default in (("tokens", 4096), ("hidden", 1024), ("inner", 512), ("experts", 64), ("topk", 4), ("steps", 8)):
        a.add_argument("--" + name, type=int, default=default)
    a.add_argument("--rate", type=float, default=0.04)
    a = a.parse_args(argv)
    moe.build()
    dev, H, I, E, K = torch.device("cuda"), a.hidden, a.inner, a.experts, a.topk
    gen = torch.Generator().manual_seed(0)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen) * std).to(dev)

    W_gate = normal(H, E, std=H ** -0.5).to(torch.bfloat16)
    teacher = [quantized(normal(E, 2 * I, H, std=H ** -0.5)), quantized(normal(E, H, I, std=I ** -0.5))]
    W1, W2 = normal(E, 2 * I, H, std=H ** -0.5), normal(E, H, I, std=I ** -0.5)
    X = normal(a.tokens, H).to(torch.bfloat16)
    target = forward(X, W_gate, K, *teacher)[0].float()
    losses = []
    for step in range(a.steps):
        W1q, W2q = quantized(W1), quantized(W2)
        loss, dW1, dW2 = 0.0, None, None
        for x, t in zip(X.chunk(2), target.chunk(2)):       # two halves, summed in the 32-bit gradients
            out, saved = forward(x, W_gate, K, W1q, W2q)
            diff = out.float() - t
            loss = loss + diff.square().sum() / X.numel()
            dout = (diff * (E / K / a.tokens)).to(torch.bfloat16)
            dW1, dW2, dX = backward(dout, saved, W1q, W2q, dW1, dW2)
        for W, dW in ((W1, dW1), (W2, dW2)):                 # a step of a given length, whatever the sizes
            W -= a.rate * W.norm() / dW.norm() * dW
        losses.append(float(loss))
        print(f"step {step}: loss {losses[-1]:.5f}, |dX| {float(dX.float().norm()):.5f}")

    W1q, W2q = quantized(W1), quantized(W2)
    few = X[:8].contiguous()
    one = moe.moe_layer(few, W_gate, K, *W1q, *W2q)
    batch, _ = forward(few, W_gate, K, W1q, W2q)
    off = float((one.out.float() - batch.float()).norm() / batch.float().norm())
    print(f"8 tokens in one launch against the batch path: relative difference {off:.5f}")
    return losses, off


if __name__ == "__main__":
    main()
