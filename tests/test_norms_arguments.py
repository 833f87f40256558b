"""Calls of the norms that no result can be right for: refused, with what is wrong."""
import pytest
import torch

import combine_moe_route_02_gb300 as moe
from test_experts import A, B, C, D, F, INVALID, L, dev, gpu, normal  # noqa: F401
from test_norms import F32, weight


def test_the_stream_and_the_normed_rows_are_not_one_tensor(L):  # noqa: F811
    """S may be X and Y may be X, but not both."""
    assert L.moe_rms_norm(A, F, B, 0, 1e-6, 4, 256, A, A, None, None, 0, D, None) == INVALID
    assert L.moe_rms_norm(A, F, B, 0, 1e-6, 4, 256, F, F, None, None, 0, D, None) == INVALID
    assert L.moe_rms_norm(A, F, B, 0, 1e-6, 4, 256, C, C, None, None, 0, D, None) == INVALID


def test_workspace_of_the_longest_lists(L):  # noqa: F811
    one = L.moe_grad_norm_workspace_size(1)
    for n in (2 ** 31 - 1024, 2 ** 31 - 1023, 2 ** 31 - 1):
        assert L.moe_grad_norm_workspace_size(n) == -(-n // 1024) * one


@gpu
def test_no_stale_stream_without_a_residual(dev):  # noqa: F811
    """Without a residual the stream is X itself: another tensor of `out` would stay what it was."""
    x, w = normal((5, 256), 1, dev), weight(256, F32, dev)
    y, s, r = torch.empty_like(x), torch.zeros_like(x), torch.empty(5, device=dev)
    with pytest.raises(ValueError, match="S"):
        moe.rms_norm(x, w, out=moe.RMSNorm(y, None, None, s, r))
    for own in (x, None):
        out = moe.rms_norm(x, w, out=moe.RMSNorm(y, None, None, own, r))
        assert torch.equal(out.Y, moe.rms_norm(x, w).Y) and out.S is own


@gpu
def test_clipping_into_another_gradient_is_refused(dev):  # noqa: F811
    a, b = torch.ones(100, device=dev), torch.ones(100, device=dev)
    with pytest.raises(ValueError, match="out"):
        moe.clip_grad_norm([a, b], 1.0, out=[b, a])
    with pytest.raises(ValueError, match="out"):
        moe.clip_grad_norm([a, b], 1.0, out=[torch.empty_like(a), a])
    moe.clip_grad_norm([a, b], 1.0, out=[a, torch.empty_like(b)])           # its own place is allowed
    e = torch.empty(0, device=dev)
    moe.clip_grad_norm([a, e, e], 1.0, out=[a, e, e])
