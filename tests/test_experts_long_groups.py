"""Weight gradients of bf16 type from groups of many rows.  All numbers are positive, so that what a sum loses in one
direction shows: the tensor cores cut where they accumulate.

A segment of 16384 rows goes into one accumulator, 16 rows to a step: it is cut 1024 times by at most 2^-23 of what it
has reached, with 8 steps' worth inside one; the segments are added in 32 bits, rounding to nearest.  One rounding to
bf16, half a step."""
import pytest
import torch

import combine_moe_route_02_gb300 as moe
import experts_ref as ref

SEGMENT = 16384


def positive(shape, seed, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev).abs().to(torch.float8_e4m3fn)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,rows,cols", [
    ([(1 << 20) + 77], 16, 128),
    # long and short groups in turn, ends of segments met exactly and missed by one, two tiles each way
    ([3 * SEGMENT, 5, 0, SEGMENT + 1, SEGMENT, 40000, 2 * SEGMENT - 1, 300, 70001], 264, 384),
    # more tiles than the pairs of a GPU hold at a time, most of them long
    ([20000, 17000, 100, 33000] * 6, 520, 1024),
])
@pytest.mark.parametrize("add", [False, True])
def test_bf16_gradients_of_long_groups(counts, rows, cols, add):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    moe.build()
    dev = torch.device("cuda")
    R = sum(counts)
    x, dY = positive((R, cols), 1, dev), positive((R, rows), 2, dev).to(torch.bfloat16)
    xs, off = torch.ones((R, cols // 128), device=dev), ref.offsets_of(counts, dev)
    base = torch.rand((len(counts), rows, cols), device=dev) * 100 if add else None
    st = torch.zeros(1, dtype=torch.int32, device=dev)

    def call():
        return moe.expert_wgrad(dY, x.view(torch.uint8), xs, off, dtype=torch.bfloat16, add=base, status=st)

    dW = call()
    assert st.item() == 0, moe.status_string(st.item())
    for _ in range(5):
        assert torch.equal(call().view(torch.int16), dW.view(torch.int16))
    at = 0
    for e, c in enumerate(counts):
        want = base[e].double() if add else torch.zeros((rows, cols), dtype=torch.float64, device=dev)
        for a in range(at, at + c, 1 << 16):
            z = min(a + (1 << 16), at + c)
            want += dY[a:z].double().T @ x[a:z].double()
        segments = -(-c // SEGMENT)
        steps = min(c, SEGMENT) / 16 + 8
        bound = want * (2.0 ** -8 + steps * 2.0 ** -23 + (segments + add) * 2.0 ** -24)
        ok = (dW[e].double() - want).abs() <= bound
        assert bool(ok.all()), (e, c, float(((dW[e].double() - want).abs() / bound).max()))
        at += c
