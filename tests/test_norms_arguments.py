"""Calls of the norms that no result can be right for: refused, with what is wrong."""
from test_experts import A, B, C, D, F, INVALID, L  # noqa: F401
from test_norms import BF16, F32, weight


def test_the_stream_and_the_normed_rows_are_not_one_tensor(L):  # noqa: F811
    """S may be X and Y may be X, but not both."""
    assert L.moe_rms_norm(A, F, B, 0, 1e-6, 4, 256, A, A, None, None, 0, D, None) == INVALID
    assert L.moe_rms_norm(A, F, B, 0, 1e-6, 4, 256, F, F, None, None, 0, D, None) == INVALID
    assert L.moe_rms_norm(A, F, B, 0, 1e-6, 4, 256, C, C, None, None, 0, D, None) == INVALID


def test_workspace_of_the_longest_lists(L):  # noqa: F811
    one = L.moe_grad_norm_workspace_size(1)
    for n in (2 ** 31 - 1024, 2 ** 31 - 1023, 2 ** 31 - 1):
        assert L.moe_grad_norm_workspace_size(n) == -(-n // 1024) * one
