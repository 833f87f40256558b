"""examples/moe_mlp.py: the experts' kernels together, as a training step and as a few-token layer; and that
step's gradients against the formulas in 64 bits, rounded where the kernels round."""
import importlib.util
import os

import pytest
import torch

import combine_moe_route_02_gb300 as moe
import experts_ref as ref

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_mlp.py")


def load():
    spec = importlib.util.spec_from_file_location("moe_mlp", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.gpu
def test_example_learns_and_serves():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    losses, off = load().main(["--tokens", "515", "--hidden", "256", "--inner", "128", "--experts", "8", "--topk", "2", "--steps", "6"])
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert off <= 2.0 ** -6            # as in test_moe_layer_agrees_with_the_batch_path


@pytest.mark.gpu
def test_step_gradients_against_the_formulas():
    """The whole step in 64 bits, with the values that the kernels hold in 8 bits taken from them: what is
    left is the roundings to bf16 and E4M3 on the way (relative 2^-8 / sqrt(3) and 2^-4 / sqrt(3) each, in norm)."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    moe.build()
    ex, dev = load(), torch.device("cuda")
    N, H, I, E, K = 300, 256, 128, 8, 2
    g = torch.Generator().manual_seed(3)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).to(dev)

    Wg = normal(H, E, std=H ** -0.5).to(torch.bfloat16)
    W1q, W2q = ex.quantized(normal(E, 2 * I, H, std=H ** -0.5)), ex.quantized(normal(E, H, I, std=I ** -0.5))
    X, dout = normal(N, H).to(torch.bfloat16), normal(N, H).to(torch.bfloat16)
    out, saved = ex.forward(X, Wg, K, W1q, W2q)
    dW1, dW2, dX = ex.backward(dout, saved, W1q, W2q)
    d, h, w = saved
    idx = torch.repeat_interleave(torch.arange(E, device=dev), d.expert_counts.long())
    D1, D2 = ref.decode(*W1q, ref.BLK), ref.decode(*W2q, ref.BLK)
    x = ref.decode(d.X_fp8, d.X_scale, 1)
    slot = d.src_slot.long()
    tok, wr = slot // K, w.double().flatten()[slot, None]
    gu = torch.einsum("rmk,rk->rm", D1[idx], x)
    act = ref.swiglu(gu)
    dy = dout.double()[tok] * wr
    da = torch.einsum("rmk,rm->rk", D2[idx], dy)
    dgu = ref.swiglu_grad(da, gu)
    dxr = torch.einsum("rmk,rm->rk", D1[idx], dgu)
    want = {
        "out": torch.zeros((N, H), dtype=torch.float64, device=dev).index_add_(0, tok, wr * torch.einsum("rmk,rk->rm", D2[idx], act)),
        "dX": torch.zeros((N, H), dtype=torch.float64, device=dev).index_add_(0, tok, dxr),
        "dW2": torch.stack([dy[idx == e].T @ act[idx == e] for e in range(E)]),
        "dW1": torch.stack([dgu[idx == e].T @ x[idx == e] for e in range(E)]),
    }
    got = {"out": out, "dX": dX, "dW2": dW2, "dW1": dW1}
    # roundings to E4M3 behind each: the activation; dY, the kept GU and dGU; the activation; dY and GU
    eight = {"out": 1, "dX": 4, "dW2": 1, "dW1": 3}
    for k in want:
        rel = float((got[k].double() - want[k]).norm() / want[k].norm())
        assert rel <= (eight[k] ** 0.5 * 2.0 ** -4 + 4 * 2.0 ** -8) / 3 ** 0.5, (k, rel)
