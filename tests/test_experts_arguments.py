"""Arguments of the experts' calls that are no tensors: a TypeError that names the argument."""
import pytest
import torch

import combine_moe_route_02_gb300 as moe
from combine_moe_route_02_gb300 import experts


@pytest.fixture(autouse=True)
def on_cpu(monkeypatch):
    """Past the checks of device and shape, which CPU tensors do not pass."""
    real = experts._arg
    monkeypatch.setattr(experts, "_home", lambda t, name: 0)
    monkeypatch.setattr(experts, "_arg", lambda t, name, *a: t.data_ptr() if isinstance(t, torch.Tensor) else real(t, name, *a))


@pytest.mark.parametrize("bad", [None, 3, [[1]], b"codes"])
@pytest.mark.parametrize("name", ["X_fp8", "X_scale", "W_fp8", "W_scale", "expert_offsets"])
@pytest.mark.parametrize("flat", [False, True])
def test_expert_gemm(name, bad, flat):
    E = 1 if flat else 2
    if name == "expert_offsets" and bad is None and flat:
        return                               # one group without offsets: allowed
    a = dict(X_fp8=torch.zeros((4, 256), dtype=torch.uint8), X_scale=torch.ones((4, 2)),
             W_fp8=torch.zeros((E, 128, 256), dtype=torch.uint8), W_scale=torch.ones((E, 1, 2)),
             expert_offsets=torch.zeros(E + 1, dtype=torch.int32))
    if flat:
        a["W_fp8"], a["W_scale"] = a["W_fp8"][0], a["W_scale"][0]
    a[name] = bad
    want = ValueError if name == "expert_offsets" and bad is None else TypeError
    with pytest.raises(want, match=name):
        moe.expert_gemm(**a)
