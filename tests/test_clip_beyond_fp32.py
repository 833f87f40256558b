"""The norm of all gradients at the upper end of fp32, and beyond it: there the norm that comes back is infinite, and as with
any norm that is not finite the tensors are left as they are."""
import math

import pytest
import torch

import combine_moe_route_02_gb300 as moe
from test_experts import dev, gpu  # noqa: F401
from test_norms import BF16, F32, NORM_TOL, check_clip, exact_norm, tensors


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_norm_just_below_the_largest_number(dev, dtype):  # noqa: F811
    grads = tensors([70000, 33], [dtype, F32], 5, dev, 0.5)
    grads = [t * 1e36 for t in grads]                        # sqrt(70033) * 0.5e36 = 1.3e38
    norm = exact_norm(grads)
    assert 1e38 < norm < 2e38
    assert abs(float(moe.grad_norm(grads)) - norm) <= NORM_TOL * norm
    check_clip([t.clone() for t in grads], norm / 4)
    check_clip(grads, norm / 4, out=[torch.empty_like(t) for t in grads])


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("most", [1e-3, 1.0, 1e30, 3e38])
def test_finite_gradients_whose_norm_is_beyond_fp32(dev, dtype, most):  # noqa: F811
    grads = [t * 3e37 for t in tensors([70000, 33], [dtype, F32], 5, dev, 0.5)]
    assert all(bool(t.isfinite().all()) for t in grads) and 3.9e39 < exact_norm(grads) < 4.1e39
    assert float(moe.grad_norm(grads)) == math.inf
    before = [t.clone() for t in grads]
    out = [torch.zeros_like(t) for t in grads]
    assert float(moe.clip_grad_norm(grads, most, out=out)) == math.inf
    assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(grads, before, out))
    assert float(moe.clip_grad_norm(grads, most)) == math.inf
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
