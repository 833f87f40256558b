"""The value checks of tests/test_experts.py once more, in a form that a NaN fails: a comparison with one is false, so
"no difference is above its bound" lets a NaN pass, "every difference is within its bound" does not.  Where the
experts' results go wrong (an accumulator nobody wrote, a scale byte 255, the next group's rows in a tile) a NaN is
the likely sign."""
import pytest
import torch

import combine_moe_route_02_gb300 as moe
import experts_ref as ref
import test_experts as checks
from test_experts import dev  # noqa: F401  (the fixture)


def within(got, want, slack, dtype=None):
    """|got - want| <= half a step of the result's type + slack, everywhere; a NaN on either side is not."""
    bound = want.abs() * ref.EPS[dtype or got.dtype] + slack
    ok = (got.double() - want).abs() <= bound
    assert bool(ok.all()), (int((~ok).sum()), int(got.isnan().sum()))


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    monkeypatch.setattr(checks, "within", within)


def test_a_nan_is_not_within():
    want = torch.ones(4, dtype=torch.float64)
    for got, w in ((want.float(), want), (want.to(torch.bfloat16) * (1 + 2.0 ** -8), want)):
        within(got, w, 0)
    bad = want.float()
    bad[2] = float("nan")
    for got, w, slack in ((bad, want, 1.0), (want.float(), bad.double(), 1.0), (want.float(), want, bad.double()),
                          (want.float() * 1.01, want, 0.0), (bad * float("nan"), want, float("inf"))):
        with pytest.raises(AssertionError):
            within(got, w, slack)


# on the GPU: the same tests, with the check above
test_expert_gemm = checks.test_expert_gemm
test_expert_gemm_one_group_without_offsets = checks.test_expert_gemm_one_group_without_offsets
test_expert_gemm_keeps_nan_to_its_rows = checks.test_expert_gemm_keeps_nan_and_scale_extremes_to_their_rows
test_expert_products_repeat = checks.test_expert_products_repeat_bit_for_bit
test_expert_products_are_each_others_gradients = checks.test_expert_products_are_each_others_gradients
test_expert_wgrad = checks.test_expert_wgrad
test_expert_wgrad_long_groups = checks.test_expert_wgrad_long_groups_keep_32_bits
test_swiglu_backward_bf16 = checks.test_swiglu_backward
test_moe_layer = checks.test_moe_layer
test_moe_layer_with_common_units = checks.test_moe_layer_with_common_units
test_moe_layer_bias_residual_and_in_place = checks.test_moe_layer_bias_residual_and_in_place


def codes_within(codes, scale, want, err):
    got = ref.decode(codes, scale, 1)
    bound = checks.quant_slack(want, err)
    ok = (got - want).abs() <= bound
    assert bool(ok.all()), (int((~ok).sum()), int(got.isnan().sum()))


@pytest.mark.gpu
@pytest.mark.parametrize("R,I", [(1, 128), (2, 256), (3, 384), (33, 128), (1001, 640)])
@pytest.mark.parametrize("fmt,gf", [("fp32", "ue8m0"), ("ue8m0", "fp32")])
def test_activation_codes(dev, R, I, fmt, gf):  # noqa: F811
    """The bounds of test_swiglu and test_swiglu_backward."""
    gu = checks.normal((R, 2 * I), R + I, dev, 3.0)
    h = moe.swiglu(gu, scale_format=fmt)
    a = ref.swiglu(gu.double())
    codes_within(h.A_fp8, h.A_scale, a, a.abs() * (2.0 ** -21 + gu.double()[:, :I].abs() * 2.0 ** -22))
    codes_within(h.GU_fp8, h.GU_scale, gu.double(), torch.zeros_like(gu, dtype=torch.float64))

    k8, ks = ref.encode_rows(checks.normal((R, 2 * I), R + I, dev, 2.0), gf)
    dA = checks.normal((R, I), 3, dev)
    r = moe.swiglu_backward(dA, k8, ks, scale_format=fmt)
    gu, da = ref.decode(k8, ks, 1), dA.double()
    g, u = gu.chunk(2, -1)
    unit = 2.0 ** -20 + torch.cat([g, g], 1).abs() * 2.0 ** -21
    err = unit * torch.cat([da.abs() * u.abs() * (1 + g.abs()), da.abs() * g.abs()], 1)
    codes_within(r.dGU_fp8, r.dGU_scale, ref.swiglu_grad(da, gu), err)
