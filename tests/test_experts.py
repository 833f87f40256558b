"""The experts: E4M3 products over ragged groups, their weight gradients, the gated
activation, the weight quantiser and the few-token layer, against the formulas in 64
bits (tests/experts_ref.py).

Tolerances count roundings.  A result of bf16 type is off by at most half a step, 2^-8 of
its value; a sum of n products held in 32 bits by at most 2^-23 of the sum of the
products' magnitudes for each step of the accumulation (2^-23 and not 2^-24, since the
tensor cores may cut where they could round), with 16 or 32 products to a step and 8
steps' worth inside one.
"""
import ctypes

import pytest
import torch

import combine_moe_route_02_gb300 as moe
import experts_ref as ref
import moe_inputs as mi

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
A, B, C, D, F = (0x10000 * i for i in range(1, 6))   # aligned fake addresses, never dereferenced


# ------------------------------------------------------------------ on the CPU: refusals

@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


def gemm(L, X=A, xs=B, xf=0, W=C, ws=D, wf=0, off=A, R=16, E=4, rows=256, cols=128, t=0, Y=F):
    return L.moe_expert_gemm(X, xs, xf, W, ws, wf, off, R, E, rows, cols, t, Y, None, None)


def test_expert_gemm_refusals(L):
    assert gemm(L, R=0) == OK
    for bad in (dict(E=0), dict(E=257), dict(R=-1), dict(R=2 ** 31), dict(rows=0), dict(cols=0), dict(xf=2), dict(wf=-1),
                dict(rows=2 ** 18 + 16), dict(cols=2 ** 18 + 128), dict(R=2 ** 31 - 2, rows=2 ** 18),
                dict(cols=192), dict(rows=200), dict(off=None), dict(X=None), dict(xs=None), dict(W=None),
                dict(ws=None), dict(Y=None), dict(t=1, rows=192), dict(t=1, cols=136)):
        assert gemm(L, **bad) == INVALID, bad
    for bad in (dict(X=A + 8), dict(W=A + 4), dict(Y=A + 2), dict(xs=A + 2), dict(ws=A + 1), dict(off=A + 2)):
        assert gemm(L, **bad) == MISALIGNED, bad


def wgrad(L, dY=A, X=B, xs=C, xf=0, off=A, R=16, E=4, rows=64, cols=128, add=None, dW=F, bf16=0):
    return L.moe_expert_wgrad(dY, X, xs, xf, off, R, E, rows, cols, add, dW, bf16, None, None)


def test_expert_wgrad_refusals(L):
    for bad in (dict(E=0), dict(E=257), dict(R=-1), dict(R=2 ** 31), dict(rows=0), dict(rows=60), dict(cols=64), dict(rows=2 ** 18 + 8),
                dict(cols=2 ** 18 + 128), dict(xf=3),
                dict(off=None), dict(dY=None), dict(X=None), dict(xs=None), dict(dW=None), dict(dW=None, R=0),
                dict(add=F, dW=F, bf16=1)):
        assert wgrad(L, **bad) == INVALID, bad
    for bad in (dict(dY=A + 2), dict(X=A + 8), dict(dW=A + 4), dict(add=A + 4), dict(xs=A + 3), dict(off=A + 1)):
        assert wgrad(L, **bad) == MISALIGNED, bad


def test_swiglu_refusals(L):
    def f(GU=A, R=8, I=128, Aq=B, As=C, K=None, Ks=None, fmt=0):
        return L.moe_swiglu(GU, R, I, Aq, As, K, Ks, fmt, None)

    assert f(R=0) == OK
    for bad in (dict(GU=None), dict(I=0), dict(I=192), dict(R=2 ** 30, I=2 ** 14), dict(R=-1), dict(Aq=None), dict(As=None), dict(fmt=2), dict(K=D), dict(Ks=D)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(GU=A + 2), dict(Aq=A + 8), dict(As=A + 2), dict(K=A + 8, Ks=D), dict(K=D, Ks=A + 1)):
        assert f(**bad) == MISALIGNED, bad

    def g(dA=A, K=B, Ks=C, kf=0, R=8, I=128, dGU=D, Q=None, Qs=None, fmt=0):
        return L.moe_swiglu_backward(dA, K, Ks, kf, R, I, dGU, Q, Qs, fmt, None, None)

    assert g(R=0) == OK
    for bad in (dict(dA=None), dict(K=None), dict(Ks=None), dict(kf=2), dict(fmt=2), dict(I=64), dict(R=-1), dict(dGU=None),
                dict(Q=F), dict(Qs=F)):
        assert g(**bad) == INVALID, bad
    for bad in (dict(dA=A + 2), dict(K=A + 8), dict(Ks=A + 2), dict(dGU=A + 8), dict(Q=F + 8, Qs=C), dict(Q=F, Qs=A + 2)):
        assert g(**bad) == MISALIGNED, bad


def test_quantize_weight_refusals(L):
    def f(W=A, E=2, rows=64, cols=64, q=B, s=C, fmt=0):
        return L.moe_quantize_weight(W, E, rows, cols, q, s, fmt, None)

    for bad in (dict(W=None), dict(q=None), dict(s=None), dict(E=0), dict(E=257), dict(rows=0), dict(rows=2 ** 22 + 1),
                dict(cols=0), dict(fmt=2)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(cols=60), dict(W=A + 8), dict(q=A + 8), dict(s=A + 2)):
        assert f(**bad) == MISALIGNED, bad


def test_moe_layer_refusals(L):
    ws_bytes = L.moe_layer_workspace_size(4, 256, 128, 8, 2)
    assert ws_bytes > 0

    def f(X=A, Wg=B, W1=C, s1=D, W2=F, s2=A, fmt=0, res=None, N=4, H=256, I=128, E=8, K=2, idx=A, w=B, out=C, ws=A, n=ws_bytes):
        return L.moe_layer(X, Wg, None, W1, s1, W2, s2, fmt, res, N, H, I, E, K, 1, idx, w, out, None, ws, n, None)

    assert f(N=0) == OK
    assert f(N=65) == UNSUPPORTED
    for bad in (dict(N=-1), dict(H=0), dict(H=192), dict(H=65536 + 128), dict(I=64), dict(E=0), dict(E=257), dict(K=0),
                dict(K=9), dict(K=17, E=32), dict(fmt=2), dict(X=None), dict(Wg=None), dict(W1=None), dict(s1=None),
                dict(W2=None), dict(s2=None), dict(idx=None), dict(w=None), dict(out=None)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(X=A + 2), dict(Wg=A + 2), dict(W1=A + 8), dict(W2=A + 8), dict(s1=A + 2), dict(s2=A + 2), dict(res=A + 2),
                dict(out=A + 8), dict(idx=A + 2), dict(w=A + 2), dict(ws=A + 16)):
        assert f(**bad) == MISALIGNED, bad
    assert f(ws=None) == WORKSPACE
    assert f(n=ws_bytes - 1) == WORKSPACE
    assert L.moe_layer_workspace_size(0, 256, 128, 8, 2) == 0
    assert L.moe_layer_workspace_size(65, 256, 128, 8, 2) == 0
    assert L.moe_layer_workspace_size(1, 256, 100, 8, 2) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x8, xs = torch.zeros((4, 256), dtype=torch.uint8), torch.ones((4, 2))
    W, ws = torch.zeros((2, 128, 256), dtype=torch.uint8), torch.ones((2, 1, 2))
    off = torch.tensor([0, 1, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        moe.expert_gemm(x8, xs, W, ws, off)
    with pytest.raises(ValueError, match="columns"):
        moe.expert_gemm(x8, xs, W, ws, off, transpose=True)
    with pytest.raises(ValueError, match="CUDA"):
        moe.expert_wgrad(torch.zeros((4, 128), dtype=torch.bfloat16), x8, xs, off)
    with pytest.raises(TypeError, match="dtype"):
        moe.expert_wgrad(torch.zeros((4, 128), dtype=torch.bfloat16), x8, xs, off, dtype=torch.float16)
    with pytest.raises(ValueError, match="scale_format"):
        moe.swiglu(torch.zeros((4, 256), dtype=torch.bfloat16), scale_format="e4m3")
    with pytest.raises(ValueError, match="CUDA"):
        moe.swiglu(torch.zeros((4, 256), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        moe.quantize_weight(torch.zeros((4, 256), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_layer(torch.zeros((1, 256), dtype=torch.bfloat16), torch.zeros((256, 2), dtype=torch.bfloat16), 1, W, ws, W, ws)


def test_reference_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    gu = torch.randn((3, 16), generator=g, dtype=torch.float64) * 2
    da = torch.randn((3, 8), generator=g, dtype=torch.float64)
    d, h = ref.swiglu_grad(da, gu), 1e-6
    for j in range(16):
        step = torch.zeros_like(gu)
        step[:, j] = h
        diff = (da * (ref.swiglu(gu + step) - ref.swiglu(gu - step))).sum(-1) / (2 * h)
        assert torch.allclose(diff, d[:, j], rtol=1e-7, atol=1e-9)


def test_reference_codec_against_torch():
    t = ref.e4m3_table()
    torch_values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.isnan(t), torch.isnan(torch_values))
    assert torch.equal(t.nan_to_num(0), torch_values.nan_to_num(0))
    x = torch.randn(4096, generator=torch.Generator().manual_seed(1)).double() * 40
    assert torch.equal(ref.round_e4m3(x)[0], x.float().clamp(-448, 448).to(torch.float8_e4m3fn).double())


# ------------------------------------------------------------------ on the GPU

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    moe.build()
    return torch.device("cuda")


def normal(shape, seed, dev, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).to(dev)


def status_word(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


def within(got, want, slack, dtype=None):
    """|got - want| <= half a step of the result's type + slack, everywhere."""
    t = want.abs() * ref.EPS[dtype or got.dtype] + slack
    over = (got.double() - want).abs() > t
    assert not over.any(), (int(over.sum()), float(((got.double() - want).abs() / t.clamp_min(1e-300)).max()))


def acc_slack(n, per_step, magnitudes):
    return (n / per_step + 8) * 2.0 ** -23 * magnitudes


COUNTS = [
    [1],                            # one row
    [0, 3, 0, 1, 0],                # empty groups at both ends
    [16, 17, 15, 224, 225, 1],      # around the tile sizes
    [449, 0, 31, 700],
    [0, 0, 0],                      # no rows in any group (the buffer has some)
]


@gpu
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("rows,cols,transpose,xf,wf", [
    (128, 128, False, "fp32", "fp32"),
    (16, 128, False, "ue8m0", "fp32"),      # a sliver of an output tile
    (272, 640, False, "fp32", "ue8m0"),     # five blocks: the scales' words are not whole
    (400, 1024, False, "ue8m0", "ue8m0"),
    (128, 16, True, "fp32", "fp32"),
    (640, 272, True, "ue8m0", "ue8m0"),
    (1024, 144, True, "fp32", "ue8m0"),
    (272, 2176, False, "fp32", "ue8m0"),    # more blocks than the scales are gathered at a time
    (2304, 528, True, "ue8m0", "fp32"),
])
def test_expert_gemm(dev, counts, rows, cols, transpose, xf, wf):
    E, R = len(counts), sum(counts) + 5      # five rows of no group
    red, n = (rows, cols) if transpose else (cols, rows)
    x8, xs = ref.encode_rows(normal((R, red), 1, dev) * torch.exp2(torch.randint(-9, 9, (R, 1), generator=torch.Generator().manual_seed(2))).to(dev), xf)
    W8, ws = ref.encode_weight(normal((E, rows, cols), 3, dev, 0.05), wf)
    off = ref.offsets_of(counts, dev)
    st = status_word(dev)
    out = torch.full((R, n), 7.0, dtype=torch.bfloat16, device=dev)
    y = moe.expert_gemm(x8, xs, W8, ws, off, transpose=transpose, out=out, status=st)
    assert st.item() == 0
    xd, Wd = ref.decode(x8, xs, 1), ref.decode(W8, ws, ref.BLK)
    a = 0
    for e, c in enumerate(counts):
        w = Wd[e] if transpose else Wd[e].T
        within(y[a:a + c], xd[a:a + c] @ w, acc_slack(red, 32, xd[a:a + c].abs() @ w.abs()))
        a += c
    assert bool((y[a:] == 7.0).all())        # rows of no group are not touched


@gpu
def test_expert_gemm_one_group_without_offsets(dev):
    x8, xs = ref.encode_rows(normal((77, 256), 5, dev), "fp32")
    W8, ws = ref.encode_weight(normal((1, 192, 256), 6, dev), "fp32")
    y = moe.expert_gemm(x8, xs, W8, ws)
    y2 = moe.expert_gemm(x8, xs, W8[0], ws[0])
    xd, Wd = ref.decode(x8, xs, 1), ref.decode(W8, ws, ref.BLK)[0]
    within(y, xd @ Wd.T, acc_slack(256, 32, xd.abs() @ Wd.abs().T))
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))
    assert moe.expert_gemm(x8[:0], xs[:0], W8, ws).shape == (0, 192)


@gpu
@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
def test_scales_need_no_alignment_beyond_their_type(dev, fmt):
    """The same bits from scales that start one element into an allocation."""
    counts = [40, 0, 33]
    x8, xs = ref.encode_rows(normal((73, 2048), 14, dev), fmt)
    W8, ws = ref.encode_weight(normal((3, 256, 2048), 15, dev), fmt)
    off, dY = ref.offsets_of(counts, dev), normal((73, 256), 16, dev)

    def moved(t):
        big = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev)
        big[1:] = t.flatten()
        return big[1:].view(t.shape)

    y, dW = moe.expert_gemm(x8, xs, W8, ws, off), moe.expert_wgrad(dY, x8, xs, off)
    assert torch.equal(moe.expert_gemm(x8, moved(xs), W8, moved(ws), off).view(torch.int16), y.view(torch.int16))
    assert torch.equal(moe.expert_wgrad(dY, x8, moved(xs), off), dW)


@gpu
def test_expert_products_repeat_bit_for_bit(dev):
    """Uneven groups, many tiles: a wait that was missing somewhere would show as a difference."""
    g = torch.Generator().manual_seed(17)
    counts = [int(c) for c in torch.randint(0, 700, (24,), generator=g)]
    R = sum(counts)
    x8, xs = ref.encode_rows(normal((R, 1152), 18, dev), "ue8m0")
    W8, ws = ref.encode_weight(normal((24, 640, 1152), 19, dev, 0.05), "ue8m0")
    off, dY = ref.offsets_of(counts, dev), normal((R, 640), 20, dev)
    y, dW = moe.expert_gemm(x8, xs, W8, ws, off), moe.expert_wgrad(dY, x8, xs, off)
    base = torch.randn(dW.shape, generator=g).to(dev)
    half = moe.expert_wgrad(dY, x8, xs, off, dtype=torch.bfloat16)
    assert torch.equal(half, dW.to(torch.bfloat16))
    for _ in range(30):
        assert torch.equal(moe.expert_gemm(x8, xs, W8, ws, off).view(torch.int16), y.view(torch.int16))
        assert torch.equal(moe.expert_wgrad(dY, x8, xs, off), dW)
        assert torch.equal(moe.expert_wgrad(dY, x8, xs, off, add=base), base + dW)
        buf = base.clone()
        assert torch.equal(moe.expert_wgrad(dY, x8, xs, off, add=buf, out=buf), base + dW)
        assert torch.equal(moe.expert_wgrad(dY, x8, xs, off, dtype=torch.bfloat16), half)
    xd, a = ref.decode(x8, xs, 1), 0
    for e, c in enumerate(counts):
        Wd = ref.decode(W8[e], ws[e], ref.BLK)
        within(y[a:a + c], xd[a:a + c] @ Wd.T, acc_slack(1152, 32, xd[a:a + c].abs() @ Wd.abs().T))
        d = dY[a:a + c].double()
        within(dW[e], d.T @ xd[a:a + c], acc_slack(c, 16, d.abs().T @ xd[a:a + c].abs()))
        a += c


@gpu
def test_expert_gemm_is_the_same_in_every_position(dev):
    """A row's result does not depend on where its group starts or what lies around it."""
    x8, xs = ref.encode_rows(normal((300, 512), 7, dev), "ue8m0")
    W8, ws = ref.encode_weight(normal((3, 256, 512), 8, dev), "ue8m0")
    a = moe.expert_gemm(x8, xs, W8, ws, ref.offsets_of([100, 0, 200], dev))
    b = moe.expert_gemm(x8[37:150].contiguous(), xs[37:150].contiguous(), W8, ws, ref.offsets_of([63, 0, 50], dev))
    assert torch.equal(a[37:150].view(torch.int16), b.view(torch.int16))


@gpu
@pytest.mark.parametrize("transpose", [False, True])
def test_expert_gemm_keeps_nan_and_scale_extremes_to_their_rows(dev, transpose):
    R, n = 70, 256
    x8, xs = ref.encode_rows(normal((R, n), 9, dev), "ue8m0")
    W8, ws = ref.encode_weight(normal((2, n, n), 10, dev), "ue8m0")
    x8[3, 5] = 0x7F                          # NaN in a row of the first group
    x8[69] = 0x7F                            # the last row of the buffer, in no group
    xs[5], ws[1] = 255, 100                  # UE8M0's NaN; small weights
    xs[40:45] = 140
    off = ref.offsets_of([30, 39], dev)
    y = moe.expert_gemm(x8, xs, W8, ws, off, transpose=transpose)
    assert bool(y[3].isnan().all()) and bool(y[5].isnan().all())
    xd, Wd = ref.decode(x8, xs, 1), ref.decode(W8, ws, ref.BLK)
    for e, (a, b) in enumerate(((0, 30), (30, 69))):
        keep = torch.tensor([r for r in range(a, b) if r not in (3, 5)], device=dev)
        w = Wd[e] if transpose else Wd[e].T
        within(y[keep], xd[keep] @ w, acc_slack(n, 32, xd[keep].abs() @ w.abs()))


@gpu
def test_expert_bad_scales_and_offsets_are_reported(dev):
    R, n = 40, 128
    x8, xs = ref.encode_rows(normal((R, n), 11, dev), "fp32")
    W8, ws = ref.encode_weight(normal((2, n, n), 12, dev), "fp32")
    good, dY = ref.offsets_of([20, 20], dev), normal((R, n), 13, dev)
    for poison in (3.0, -1.0, 0.0, float("inf"), float("nan")):
        bad = xs.clone()
        bad[7] = poison
        st = status_word(dev)
        moe.expert_gemm(x8, bad, W8, ws, good, status=st)
        expect = moe.ERR_BAD_SCALE
        assert st.item() == expect, poison
        st.zero_()
        moe.expert_gemm(x8, xs, W8, torch.full_like(ws, 3.0), good, status=st)
        assert st.item() == expect
        st.zero_()
        moe.expert_wgrad(dY, x8, bad, good, status=st)
        assert st.item() == expect, poison
    for off in ([0, 20, 41], [-1, 20, 40], [0, 30, 20], [50, 60, 70]):
        st = status_word(dev)
        o = torch.tensor(off, dtype=torch.int32, device=dev)
        out = torch.full((R, n), 7.0, dtype=torch.bfloat16, device=dev)
        moe.expert_gemm(x8, xs, W8, ws, o, out=out, status=st)
        assert st.item() == moe.ERR_BAD_INDEX, off
        st.zero_()
        moe.expert_wgrad(dY, x8, xs, o, status=st)
        assert st.item() == moe.ERR_BAD_INDEX, off
    assert bool((out == 7.0).all())          # [50, 60, 70]: both groups outside


@gpu
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("rows,cols,xf,dtype,add", [
    (128, 256, "fp32", torch.float32, False),
    (8, 128, "ue8m0", torch.bfloat16, False),
    (200, 384, "ue8m0", torch.float32, True),
    (264, 640, "fp32", torch.bfloat16, True),
])
def test_expert_wgrad(dev, counts, rows, cols, xf, dtype, add):
    E, R = len(counts), sum(counts) + 5
    x8, xs = ref.encode_rows(normal((R, cols), 21, dev), xf)
    dY = normal((R, rows), 22, dev)
    x8[-5:], dY[-5:] = 0x7F, float("nan")    # rows of no group, right behind the last one
    off = ref.offsets_of(counts, dev)
    base = torch.randn((E, rows, cols), generator=torch.Generator().manual_seed(23)).to(dev) if add else None
    kept = base.clone() if add else None
    st = status_word(dev)
    dW = moe.expert_wgrad(dY, x8, xs, off, dtype=dtype, add=base, status=st)
    assert st.item() == 0
    xd, dYd = ref.decode(x8, xs, 1), dY.double()
    a = 0
    for e, c in enumerate(counts):
        want = dYd[a:a + c].T @ xd[a:a + c]
        slack = acc_slack(c, 16, dYd[a:a + c].abs().T @ xd[a:a + c].abs())
        if add:
            want = want + kept[e].double()
            slack = slack + 2.0 ** -24 * want.abs()
        within(dW[e], want, slack)
        a += c
    if add:
        assert torch.equal(base, kept)
        if dtype == torch.float32:           # in place, the same bits
            assert moe.expert_wgrad(dY, x8, xs, off, add=base, out=base) is base
            assert torch.equal(base, dW)


@gpu
@pytest.mark.parametrize("add", [False, True])
def test_expert_wgrad_long_groups_keep_32_bits(dev, add):
    """Groups longer than the 2048 rows that go into one accumulator.  A tensor core's sum of 2048 rows is cut
    128 times by at most 2^-23 of what it has reached, on average two thirds of the end: 1e-5 at the worst, a
    tenth of that as it comes out; segments added with rounding to nearest keep to it however long the group."""
    counts = [5000, 0, 2048, 2049, 1, 9000]
    R, rows, cols = sum(counts), 264, 256
    x8, xs = ref.encode_rows(normal((R, cols), 24, dev), "fp32")
    dY, off = normal((R, rows), 25, dev), ref.offsets_of(counts, dev)
    base = torch.randn((len(counts), rows, cols), generator=torch.Generator().manual_seed(26)).to(dev) if add else None
    dW = moe.expert_wgrad(dY, x8, xs, off, add=base)
    for _ in range(10):
        assert torch.equal(moe.expert_wgrad(dY, x8, xs, off, add=base), dW)
    if add:
        buf = base.clone()
        assert torch.equal(moe.expert_wgrad(dY, x8, xs, off, add=buf, out=buf), dW)
    xd, a = ref.decode(x8, xs, 1), 0
    for e, c in enumerate(counts):
        d = dY[a:a + c].double()
        want = d.T @ xd[a:a + c] + (base[e].double() if add else 0)
        if c:
            assert (dW[e].double() - want).norm() <= 2.0 ** -20 * want.norm()
        within(dW[e], want, acc_slack(c, 16, d.abs().T @ xd[a:a + c].abs()))
        a += c


@gpu
def test_expert_wgrad_values_at_the_edges_of_e4m3(dev):
    """Every code under scales from the smallest bf16 holds to the largest, NaN codes included: a
    product with one-hot rows gives each value back."""
    codes = torch.arange(256, dtype=torch.uint8, device=dev).view(2, 128)
    for byte in (10, 60, 127, 134, 135, 180, 245):
        x8 = codes.repeat(8, 1)                                   # 16 rows
        xs = torch.full((16, 1), byte, dtype=torch.uint8, device=dev)
        dY = torch.eye(16, dtype=torch.bfloat16, device=dev)
        finite = ((x8 & 127) != 127).all(1)
        dW = moe.expert_wgrad(dY, torch.where((x8 & 127) == 127, 0, x8), xs)[0]
        want = ref.decode(torch.where((x8 & 127) == 127, 0, x8), xs, 1)
        assert torch.equal(dW.double(), want), byte
        assert not finite.any()
        dW = moe.expert_wgrad(dY, x8, xs)[0]
        assert bool(dW[:, 127].isnan().all()) and not dW[:, :127].isnan().any(), byte


@gpu
def test_expert_wgrad_without_rows(dev):
    x8 = torch.empty((0, 256), dtype=torch.uint8, device=dev)
    xs, dY = torch.empty((0, 2), device=dev), torch.empty((0, 64), dtype=torch.bfloat16, device=dev)
    off = torch.zeros(4, dtype=torch.int32, device=dev)
    assert bool((moe.expert_wgrad(dY, x8, xs, off) == 0).all())
    add = torch.ones((3, 64, 256), device=dev)
    assert torch.equal(moe.expert_wgrad(dY, x8, xs, off, add=add), add)


@gpu
def test_expert_products_are_each_others_gradients(dev):
    """<dY, x W^T> = <dY W, x> = <dW, W> for values that E4M3 and bf16 hold exactly."""
    g = torch.Generator().manual_seed(31)
    counts = [5, 0, 130]
    R, n, k = sum(counts), 128, 256
    xv, Wv = torch.randint(-4, 5, (R, k), generator=g).to(dev), torch.randint(-4, 5, (3, n, k), generator=g).to(dev)
    dv = torch.randint(-4, 5, (R, n), generator=g).to(dev)

    def coded(v):
        return v.float().to(torch.float8_e4m3fn).view(torch.uint8)

    off = ref.offsets_of(counts, dev)
    ones_k, ones_n = torch.ones((R, k // 128), device=dev), torch.ones((R, n // 128), device=dev)
    ws = torch.ones((3, 1, 2), device=dev)
    y = torch.zeros((R, n), dtype=torch.float64, device=dev)
    e = torch.repeat_interleave(torch.arange(3, device=dev), torch.tensor(counts, device=dev))
    y = (Wv.double()[e] * xv.double()[:, None]).sum(-1)
    total = (dv.double() * y).sum()
    dW = moe.expert_wgrad(dv.to(torch.bfloat16), coded(xv), ones_k, off)
    assert (dW.double() * Wv.double()).sum() == total             # integers: exact in 32 bits
    dx = moe.expert_gemm(coded(dv), ones_n, coded(Wv), ws, off, transpose=True)
    want = (Wv.double()[e] * dv.double()[..., None]).sum(1)
    within(dx, want, 0)
    within(moe.expert_gemm(coded(xv), ones_k, coded(Wv), ws, off), y, 0)
    assert (want * xv.double()).sum() == total


def quant_slack(want, err):
    """What a value's E4M3 form may be off: half a step, and what the value itself was off (which
    may also carry it over the border to the next code)."""
    _, scale, step = ref.quant_rows(want)
    return step / 2 + 2 * err


@gpu
@pytest.mark.parametrize("R,I", [(1, 128), (2, 256), (3, 384), (33, 128), (1001, 640)])
@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
def test_swiglu(dev, R, I, fmt):
    gu = normal((R, 2 * I), R + I, dev, 3.0)
    h = moe.swiglu(gu, scale_format=fmt)
    a = ref.swiglu(gu.double())
    # exp, the sum, the division and the product in 32 bits: a few units in the last place, and the
    # rounding of the exponent's argument (|g| * 2^-24 * 1.5 of the exponential)
    err = a.abs() * (2.0 ** -21 + gu.double()[:, :I].abs() * 2.0 ** -22)
    got = ref.decode(h.A_fp8, h.A_scale, 1)
    assert not ((got - a).abs() > quant_slack(a, err)).any()
    # the checkpoint is the rounding of what is there: the codes of moe_permute, bit for bit
    x8, xs = ref.encode_rows(gu, fmt)
    assert torch.equal(h.GU_fp8, x8) and torch.equal(h.GU_scale, xs)
    ident = torch.arange(R, dtype=torch.int32, device=dev).view(R, 1)
    p = moe.dispatch(torch.zeros((R, 1), dtype=torch.int32, device=dev), 1, gu, fp8=True, scale_format=fmt)
    assert torch.equal(p.row_map, ident.view(-1)) and torch.equal(p.X_fp8, x8) and torch.equal(p.X_scale, xs)
    alone = moe.swiglu(gu, keep=False, scale_format=fmt)
    assert alone.GU_fp8 is None and torch.equal(alone.A_fp8, h.A_fp8) and torch.equal(alone.A_scale, h.A_scale)


@gpu
def test_swiglu_large_and_special_values(dev):
    gu = torch.zeros((6, 256), dtype=torch.bfloat16, device=dev)
    gu[0, :128], gu[0, 128:] = -100.0, 1.0     # exp overflows: silu is -0
    gu[1, :128], gu[1, 128:] = 100.0, 2.0
    gu[2, 3] = float("nan")
    gu[3, :128], gu[3, 128:] = 3e38, 1.0
    gu[4, :128], gu[4, 128:] = 1e-30, 1e-30
    h = moe.swiglu(gu, scale_format="fp32")
    v = ref.decode(h.A_fp8, h.A_scale, 1)
    assert bool((v[0] == 0).all()) and bool((v[4] == 0).all()) and bool((v[5] == 0).all())
    assert bool(((v[1] - 200).abs() <= 200 * 2.0 ** -4).all())
    assert v[2, 3].isnan() and not v[2, :3].isnan().any() and not v[2, 4:].isnan().any()
    assert bool(((v[3] / 3e38 - 1).abs() <= 2.0 ** -4).all())
    kept = ref.decode(h.GU_fp8, h.GU_scale, 1)
    assert kept[2, 3].isnan() and int(kept.isnan().sum()) == 1
    b = moe.swiglu_backward(torch.ones((6, 128), dtype=torch.bfloat16, device=dev), h.GU_fp8, h.GU_scale)
    assert int(b.dGU.isnan().sum()) == 2       # the NaN's gate and up gradients
    assert bool((b.dGU[0] == 0).all())


@gpu
@pytest.mark.parametrize("R,I", [(1, 128), (2, 256), (35, 384), (1001, 128)])
@pytest.mark.parametrize("gf,fmt", [("fp32", "ue8m0"), ("ue8m0", "fp32")])
def test_swiglu_backward(dev, R, I, gf, fmt):
    k8, ks = ref.encode_rows(normal((R, 2 * I), R + I, dev, 2.0), gf)
    dA = normal((R, I), 3, dev)
    st = status_word(dev)
    r = moe.swiglu_backward(dA, k8, ks, scale_format=fmt, status=st)
    assert st.item() == 0
    gu, da = ref.decode(k8, ks, 1), dA.double()
    want = ref.swiglu_grad(da, gu)
    g, u = gu.chunk(2, -1)
    # as for the forward pass; the gate's gradient is a sum of two terms that may cancel
    unit = 2.0 ** -20 + torch.cat([g, g], 1).abs() * 2.0 ** -21
    err = unit * torch.cat([da.abs() * u.abs() * (1 + g.abs()), da.abs() * g.abs()], 1)
    within(r.dGU, want, err)
    assert not ((ref.decode(r.dGU_fp8, r.dGU_scale, 1) - want).abs() > quant_slack(want, err)).any()
    only = moe.swiglu_backward(dA, k8, ks, fp8=False)
    assert only.dGU_fp8 is None and torch.equal(only.dGU.view(torch.int16), r.dGU.view(torch.int16))
    only = moe.swiglu_backward(dA, k8, ks, bf16=False, scale_format=fmt)
    assert only.dGU is None and torch.equal(only.dGU_fp8, r.dGU_fp8) and torch.equal(only.dGU_scale, r.dGU_scale)


@gpu
def test_swiglu_backward_reports_bad_scales(dev):
    k8, ks = ref.encode_rows(normal((4, 256), 1, dev), "fp32")
    ks[2, 1] = 0.3
    st = status_word(dev)
    moe.swiglu_backward(normal((4, 128), 2, dev), k8, ks, status=st)
    assert st.item() == moe.ERR_BAD_SCALE


@gpu
@pytest.mark.parametrize("shape", [(1, 1, 8), (2, 128, 128), (3, 129, 136), (1, 300, 1000), (5, 16, 264)])
@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
def test_quantize_weight(dev, shape, fmt):
    W = normal(shape, 41, dev, 0.02)
    W[0, 0, :8] = torch.tensor([0.0, -0.0, 448.0, -448.0, 1e-30, 3e38, float("nan"), 1.0], dtype=torch.bfloat16)
    if shape[0] > 1:
        W[1] = 0                                # the smallest scale
    q, s = moe.quantize_weight(W, scale_format=fmt)
    want_q, want_s = ref.encode_weight(W.nan_to_num(0.0), fmt)
    nan = W.isnan()
    assert torch.equal(s, want_s)
    assert torch.equal(q[~nan], want_q[~nan]) and bool(((q[nan] & 127) == 127).all())
    q2, s2 = moe.quantize_weight(W[0].contiguous(), scale_format=fmt)
    assert torch.equal(q2, q[0]) and torch.equal(s2, s[0])


# ------------------------------------------------------------------ the few-token layer

def layer_inputs(N, H, I, E, K, fmt, dev, seed=0):
    X, Wg = normal((N, H), seed + 1, dev), normal((H, E), seed + 2, dev, H ** -0.5)
    W1, s1 = ref.encode_weight(normal((E, 2 * I, H), seed + 3, dev, H ** -0.5), fmt)
    W2, s2 = ref.encode_weight(normal((E, H, I), seed + 4, dev, I ** -0.5), fmt)
    return X, Wg, W1, s1, W2, s2


def check_layer(r, X, Wg, W1, s1, W2, s2, K, bias=None, renorm=True, residual=None):
    N, H = X.shape
    E, I = W1.shape[0], W2.shape[2]
    logits = X.double() @ Wg.double() + (0 if bias is None else bias.double())
    top, order = torch.sort(logits, dim=1, descending=True, stable=True)
    if E > K:                                   # the choice is the router's where 32 bits can tell
        assert bool((top[:, :-1] - top[:, 1:])[:, :K].min() > 1e-5), "choose another seed"
    assert torch.equal(r.topk_idx.long(), order[:, :K])
    p = torch.softmax(logits, 1).gather(1, order[:, :K])
    if renorm:
        p = p / p.sum(1, keepdim=True)
    assert (r.topk_w.double() - p).abs().max() <= 1e-5
    w = r.topk_w.double()
    xq = ref.quant_rows(X.double())[0]
    want = torch.zeros((N, H), dtype=torch.float64, device=X.device)
    slack = torch.zeros_like(want)
    for n in range(N):
        for k in range(K):
            e = int(order[n, k])
            D1, D2 = ref.decode(W1[e], s1[e], ref.BLK), ref.decode(W2[e], s2[e], ref.BLK)
            gu, mag = D1 @ xq[n], D1.abs() @ xq[n].abs()
            g, u = gu.chunk(2)
            dgu = acc_slack(H, 32, mag)
            a = ref.swiglu(gu[None])[0]
            # first order: |da| <= 1.1 |u| dg + |silu| du, and the activation's own roundings
            da = 1.1 * u.abs() * dgu[:I] + g.abs() * dgu[I:] + a.abs() * (2.0 ** -21 + g.abs() * 2.0 ** -22)
            aq, scale, step = (t[0] for t in ref.quant_rows(a[None]))
            # a value within da of the border between two codes may become either; a block whose
            # maximum is that near to where its scale doubles, one coarser rounding anywhere
            border = ((a / step - torch.floor(a / step)) - 0.5).abs() * step <= da + 1e-12
            amax = a.abs().unflatten(0, (-1, 128)).amax(-1)
            near = ((amax * (1 + 1e-4) / 448).log2().ceil() != (amax * (1 - 1e-4) / 448).log2().ceil()).repeat_interleave(128)
            off = step * border + 2 * step * near
            y, ymag = D2 @ aq, D2.abs() @ aq.abs()
            want[n] += w[n, k] * y
            slack[n] += w[n, k] * (D2.abs() @ off + acc_slack(I, 32, ymag) + 2.0 ** -22 * ymag)
    if residual is not None:
        want = want + residual.double()
    within(r.out, want, slack + 2.0 ** -22 * want.abs())


@gpu
@pytest.mark.parametrize("N,H,I,E,K,fmt", [
    (1, 128, 128, 1, 1, "fp32"),
    (1, 256, 128, 8, 2, "ue8m0"),
    (5, 384, 256, 6, 4, "fp32"),        # E and K that do not divide anything
    (9, 256, 128, 2, 2, "ue8m0"),       # more than a group of 8 tokens on every expert
    (33, 256, 384, 16, 3, "fp32"),
    (64, 128, 128, 4, 4, "ue8m0"),      # all tokens on all experts
    (64, 256, 128, 64, 8, "fp32"),
    (3, 2176, 256, 8, 2, "ue8m0"),      # a reduction wider than a stage
    (2, 256, 2304, 4, 2, "fp32"),       # and in the second product
    (17, 512, 128, 256, 16, "fp32"),    # the most experts and choices
    (2, 4096, 128, 40, 5, "ue8m0"),
])
def test_moe_layer(dev, N, H, I, E, K, fmt):
    t = layer_inputs(N, H, I, E, K, fmt, dev)
    st = status_word(dev)
    r = moe.moe_layer(t[0], t[1], K, *t[2:], status=st)
    assert st.item() == 0, moe.status_string(st.item())
    check_layer(r, *t, K)


@gpu
@pytest.mark.parametrize("H,I,E", [
    (768, 384, 256),      # some 10600 units of weights in each product: the last are common to the CTAs
    (512, 640, 160),      # 12000 and 4800: in the first product only
])
def test_moe_layer_with_common_units(dev, H, I, E):
    """Which CTA takes a common unit changes nothing, and the count of them starts anew with every call."""
    N, K = 64, 8
    t = layer_inputs(N, H, I, E, K, "ue8m0", dev, seed=90)
    ws = moe.layer_workspace(N, H, I, E, K)
    st = status_word(dev)
    first = moe.moe_layer(t[0], t[1], K, *t[2:], workspace=ws, status=st)
    check_layer(first, *t, K)
    for rep in range(30):
        r = moe.moe_layer(t[0], t[1], K, *t[2:], workspace=ws, status=st)
        assert torch.equal(r.out.view(torch.int16), first.out.view(torch.int16)), rep
    assert st.item() == 0, moe.status_string(st.item())


@gpu
@pytest.mark.parametrize("renorm", [True, False])
def test_moe_layer_bias_residual_and_in_place(dev, renorm):
    t = layer_inputs(7, 256, 128, 16, 3, "fp32", dev, seed=50)
    bias = torch.linspace(-1, 1, 16, device=dev)
    res = normal((7, 256), 60, dev)
    r = moe.moe_layer(t[0], t[1], 3, *t[2:], bias=bias, renorm=renorm, residual=res)
    check_layer(r, *t, 3, bias, renorm, res)
    buf = res.clone()
    again = moe.moe_layer(t[0], t[1], 3, *t[2:], bias=bias, renorm=renorm, residual=buf,
                          out=moe.LayerOut(buf, torch.empty_like(r.topk_idx), torch.empty_like(r.topk_w)))
    assert again.out is buf and torch.equal(buf.view(torch.int16), r.out.view(torch.int16))


@gpu
def test_moe_layer_ties_nan_and_one_busy_expert(dev):
    X, Wg, W1, s1, W2, s2 = layer_inputs(12, 256, 128, 8, 2, "fp32", dev, seed=70)
    r = moe.moe_layer(X, torch.zeros_like(Wg), 2, W1, s1, W2, s2)
    assert bool((r.topk_idx == torch.tensor([0, 1], device=dev)).all()) and bool((r.topk_w == 0.5).all())
    bias = torch.full((8,), float("nan"), device=dev)
    bias[5] = 0.0
    bias[3] = -1e30
    r = moe.moe_layer(X, Wg, 2, W1, s1, W2, s2, bias=bias)
    assert bool((r.topk_idx == torch.tensor([5, 3], device=dev)).all())
    assert bool((r.topk_w == torch.tensor([1.0, 0.0], device=dev)).all())
    X[4, 7] = float("nan")                      # a token's NaN stays in its row
    r = moe.moe_layer(X, torch.zeros_like(Wg), 2, W1, s1, W2, s2)
    assert bool(r.out[4].isnan().all()) and not r.out[:4].isnan().any() and not r.out[5:].isnan().any()


@gpu
def test_moe_layer_repeats_on_one_workspace_and_as_a_graph(dev):
    """Calls of several sizes on one workspace, back to back and from a CUDA graph, give the same bits."""
    E, I, H, K = 16, 256, 512, 4
    t = layer_inputs(32, H, I, E, K, "ue8m0", dev, seed=80)
    big = moe.layer_workspace(32, H, I, E, K)
    first = {}
    for rep in range(40):
        for n in (32, 1, 7):
            r = moe.moe_layer(t[0][:n].contiguous(), t[1], K, *t[2:], workspace=big)
            if rep == 0:
                first[n] = r
            else:
                assert torch.equal(r.out.view(torch.int16), first[n].out.view(torch.int16))
                assert torch.equal(r.topk_w, first[n].topk_w)
    assert bool((big[:256 + 4 * (E + 128) * (I // 128)] == 0).all())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x = t[0][:7].contiguous()
    with torch.cuda.stream(s):
        own = moe.layer_workspace(7, H, I, E, K)
        moe.moe_layer(x, t[1], K, *t[2:], workspace=own)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r = moe.moe_layer(x, t[1], K, *t[2:], workspace=own)
    for _ in range(3):
        r.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r.out.view(torch.int16), first[7].out.view(torch.int16))


@gpu
@pytest.mark.parametrize("n", [1, 7])
def test_moe_layer_gives_up_a_wait_and_recovers(dev, n):
    """An arrival counter that can never be reached (it wraps one short): every CTA gives up after its limit,
    the status word says so, the counters end at zero and the next call is right."""
    E, I, H, K = 16, 256, 512, 4
    t = layer_inputs(n, H, I, E, K, "fp32", dev, seed=85)
    ws = torch.zeros(moe.layer_workspace_size(n, H, I, E, K), dtype=torch.uint8, device=dev)
    ws[:4] = 255
    st = status_word(dev)
    moe.moe_layer(t[0], t[1], K, *t[2:], workspace=ws, status=st)
    assert st.item() == moe.ERR_TIMEOUT
    assert bool((ws[:256 + 4 * (E + 128) * (I // 128)] == 0).all())
    st.zero_()
    r = moe.moe_layer(t[0], t[1], K, *t[2:], workspace=ws, status=st)
    assert st.item() == 0
    check_layer(r, *t, K)


@gpu
def test_moe_layer_agrees_with_the_batch_path(dev):
    """dispatch, the two products with the activation between them, and combine: the same layer up to
    the bf16 roundings between its steps."""
    N, H, I, E, K = 48, 512, 256, 16, 4
    X, Wg, W1, s1, W2, s2 = layer_inputs(N, H, I, E, K, "ue8m0", dev, seed=90)
    r = moe.moe_layer(X, Wg, K, W1, s1, W2, s2)
    idx, w = moe.route(X, Wg, K)
    assert torch.equal(idx, r.topk_idx)
    d = moe.dispatch(idx, E, X, fp8=True, bf16=False, scale_format="ue8m0")
    h = moe.swiglu(moe.expert_gemm(d.X_fp8, d.X_scale, W1, s1, d.expert_offsets), scale_format="ue8m0")
    y = moe.expert_gemm(h.A_fp8, h.A_scale, W2, s2, d.expert_offsets)
    out = moe.combine(y, d.row_map, w)
    diff = (out.double() - r.out.double()).norm() / r.out.double().norm()
    # gate and up rounded to bf16 (2^-8 / sqrt(3) each, uniform), some E4M3 codes one step on, y and out
    assert diff <= 2.0 ** -6


@gpu
def test_experts_on_another_stream(dev):
    s = torch.cuda.Stream()
    x8, xs = ref.encode_rows(normal((200, 256), 1, dev), "fp32")
    W8, ws = ref.encode_weight(normal((1, 256, 256), 2, dev), "fp32")
    want = moe.expert_gemm(x8, xs, W8, ws)
    torch.cuda.synchronize()
    out = torch.zeros_like(want)
    s.wait_stream(torch.cuda.current_stream())
    got = moe.expert_gemm(x8, xs, W8, ws, out=out, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
