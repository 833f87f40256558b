"""examples/moe_block.py: the norm, the joined products, the combine and the clipping as a block uses them, and the
block's gradients against the formulas in 64 bits, with the values that the kernels hold in 8 bits taken from them."""
import importlib.util
import os

import pytest
import torch

import combine_moe_route_02_gb300 as moe
import experts_ref as ref

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


def load():
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    moe.build()


@pytest.mark.gpu
def test_example_runs_and_clips():
    need_gpu()
    norms, after = load().main(["--tokens", "515", "--hidden", "256", "--inner", "128", "--experts", "8", "--topk", "2", "--steps", "3", "--max-norm", "0.01"])
    assert all(n > 0.01 and n == n for n in norms)
    # the coefficient and each scaled value are rounded: 2^-24 each, and the norm of them to 34 * 2^-24 (test_norms.py),
    # twice; the coefficient's own 1e-6 beside the norm
    assert abs(after[0] - 0.01) <= 0.01 * (80 * 2.0 ** -24 + 1e-6 / norms[-1])


@pytest.mark.gpu
def test_block_gradients_against_the_formulas():
    """What is left is the roundings to bf16 and E4M3 on the way (relative 2^-8 / sqrt(3) and 2^-4 / sqrt(3) each, in
    norm, at the most)."""
    need_gpu()
    ex, dev = load(), torch.device("cuda")
    N, H, I, E, K = 300, 256, 128, 8, 2
    gen = torch.Generator().manual_seed(3)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen) * std).to(dev)

    Wg = normal(H, E, std=H ** -0.5).to(torch.bfloat16)
    W1q, W2q = ex.quantized(normal(E, 2 * I, H, std=H ** -0.5)), ex.quantized(normal(E, H, I, std=I ** -0.5))
    V1q, V2q = ex.quantized(normal(2 * I, H, std=H ** -0.5)), ex.quantized(normal(H, I, std=I ** -0.5))
    w = 1 + normal(H, std=0.2)
    x, attn, dout = (normal(N, H).to(torch.bfloat16) for _ in range(3))
    out, saved = ex.forward(x, attn, w, Wg, K, W1q, W2q, V1q, V2q)
    grads, dx = ex.backward(dout, saved, w, W1q, W2q, V1q, V2q)
    n, p, d = saved.n, saved.p, saved.d

    s = (x.double() + attn.double()).to(torch.bfloat16).double()
    rstd = (s.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    xh = s * rstd
    y = xh * w.double()
    assert (n.Y.double() - y).norm() <= 2.0 ** -8 * y.norm() and (ref.decode(n.Y_fp8, n.Y_scale, 1) - y).norm() <= 2.0 ** -4 * y.norm()
    D1, D2, B1, B2 = (ref.decode(*q, ref.BLK) for q in (W1q, W2q, V1q, V2q))
    idx = torch.repeat_interleave(torch.arange(E, device=dev), d.expert_counts.long())
    slot = d.src_slot.long()
    tok, pr = slot // K, p.double().flatten()[slot, None]
    xr, xs, do = ref.decode(d.X_fp8, d.X_scale, 1), ref.decode(n.Y_fp8, n.Y_scale, 1), dout.double()
    gu, gus = torch.einsum("rmk,rk->rm", D1[idx], xr), xs @ B1.T
    act, acts = ref.swiglu(gu), ref.swiglu(gus)
    dE = do[tok] * pr
    dgu = ref.swiglu_grad(torch.einsum("rmk,rm->rk", D2[idx], dE), gu)
    dgus = ref.swiglu_grad(do @ B2, gus)
    dY = torch.zeros((N, H), dtype=torch.float64, device=dev).index_add_(0, tok, torch.einsum("rmk,rm->rk", D1[idx], dgu)) + dgus @ B1
    dn = dY * w.double()
    want = {
        "out": s + torch.zeros_like(s).index_add_(0, tok, pr * torch.einsum("rmk,rk->rm", D2[idx], act)) + acts @ B2.T,
        "dW1": torch.stack([dgu[idx == e].T @ xr[idx == e] for e in range(E)]),
        "dW2": torch.stack([dE[idx == e].T @ act[idx == e] for e in range(E)]),
        "dV1": dgus.T @ xs, "dV2": do.T @ acts,
        "dw": (dY * xh).sum(0),
        "dx": rstd * (dn - xh * (dn * xh).mean(1, keepdim=True)) + do,
    }
    got = dict(zip(("dW1", "dW2", "dV1", "dV2", "dw"), grads), out=out, dx=dx)
    # roundings to E4M3 behind each: the activation; what goes into the down projection's gradient, the kept halves and
    # their gradient
    eight = {"out": 1, "dW1": 3, "dW2": 1, "dV1": 3, "dV2": 1, "dw": 3, "dx": 3}
    for k in want:
        rel = float((got[k].double() - want[k]).norm() / want[k].norm())
        assert rel <= (eight[k] ** 0.5 * 2.0 ** -4 + 4 * 2.0 ** -8) / 3 ** 0.5, (k, rel)
