"""The norm's gradient against differences: the formula that the tests hold the kernel to, on the CPU, and the kernel itself."""
import pytest
import torch

import combine_moe_route_02_gb300 as moe
from test_experts import dev, gpu  # noqa: F401
from test_norms import BF16, F32, U

EPS = 1e-3


def loss(s, w, dy):
    return (dy * s * (s.square().mean(1, keepdim=True) + EPS).rsqrt() * w).sum()


def formula(s, w, dy):
    r = (s.square().mean(1, keepdim=True) + EPS).rsqrt()
    xh, d = s * r, dy * w
    return r * (d - xh * (d * xh).mean(1, keepdim=True)), (dy * xh).sum(0)


def differences(s, w, dy, h=2.0 ** -20):
    """Central differences: their error is h^2 / 6 of the third derivative, some 1e-12, and 2^-53 / h of the
    loss, some 1e-8: 1e-7 is allowed."""
    out = []
    for at in (s, w):
        g = torch.empty_like(at)
        for i in range(at.numel()):
            keep = at.view(-1)[i].item()
            at.view(-1)[i] = keep + h
            up = loss(s, w, dy)
            at.view(-1)[i] = keep - h
            g.view(-1)[i] = (up - loss(s, w, dy)) / (2 * h)
            at.view(-1)[i] = keep
        out.append(g)
    return out


def inputs(H, seed):
    """Values that bf16 (s, dy) and fp32 (w) hold."""
    g = torch.Generator().manual_seed(seed)
    s, dy = (torch.randn((3, H), generator=g).to(BF16) for _ in range(2))
    return s, torch.randn(H, generator=g), dy


@pytest.mark.parametrize("H", [8, 136])
def test_formula(H):
    s, w, dy = (t.double() for t in inputs(H, H))
    for a, b in zip(differences(s, w, dy), formula(s, w, dy)):
        assert float((a - b).abs().max()) < 1e-7


@gpu
@pytest.mark.parametrize("H", [8, 136, 1192])
def test_kernel(dev, H):  # noqa: F811
    s, w, dy = inputs(H, H)
    rstd = (s.double().square().mean(1) + EPS).rsqrt()
    got = moe.rms_norm_backward(dy.to(dev), s.to(dev), w.to(dev), rstd.float().to(dev))
    s, w, dy = s.double(), w.double(), dy.double()
    dx, dw = differences(s, w, dy)
    r = rstd[:, None]
    xh, d = s * r, dy * w
    size = (d * xh).abs().mean(1, keepdim=True)
    # as in test_rms_norm_backward, and rstd's own rounding, which is in d once and in the other term three times
    slack = r * (xh.abs() * 67 * U * size + 5 * U * (d.abs() + (xh * (d * xh).mean(1, keepdim=True)).abs())) + 1e-7
    assert not ((got.dX.cpu().double() - dx).abs() > slack + 2.0 ** -8 * (dx.abs() + slack)).any()
    # three rows in as many warps or CTAs: three sums in the table or of it, the rounding of rstd, of s rstd and of the sum
    assert not ((got.dweight.cpu().double() - dw).abs() > 8 * U * (dy * xh).abs().sum(0) + 1e-7).any()
