"""Both projections with the gated activation in one launch, and the down projection's input gradient with the
activation's, against the formulas in 64 bits (tests/experts_ref.py).

Tolerances: the product's own (test_experts.py's acc_slack) carried through the activation by its derivatives, the
activation's arithmetic as in test_swiglu and test_swiglu_backward, then half a step of the result's type.
"""
import pytest
import torch

import combine_moe_route_02_gb300 as moe
import experts_ref as ref
from test_experts import A, B, C, COUNTS, D, F, INVALID, MISALIGNED, OK, L, acc_slack, dev, gpu, normal, quant_slack, status_word, within  # noqa: F401

BF16, U8 = torch.bfloat16, torch.uint8


# ------------------------------------------------------------------ on the CPU: refusals

def test_expert_swiglu_refusals(L):  # noqa: F811
    def f(X=A, xs=B, xf=0, W=C, ws=D, wf=0, off=A, R=16, E=4, H=128, I=128, Aq=F, As=B, K=None, Ks=None, fmt=0):
        return L.moe_expert_swiglu(X, xs, xf, W, ws, wf, off, R, E, H, I, Aq, As, K, Ks, fmt, None, None)

    assert f(R=0) == OK
    for bad in (dict(E=0), dict(E=257), dict(R=-1), dict(R=2 ** 31 - 1), dict(H=0), dict(H=192), dict(H=2 ** 18 + 128), dict(I=0),
                dict(I=64), dict(I=-128), dict(I=2 ** 17 + 128), dict(R=2 ** 31 - 2, I=2 ** 17), dict(xf=2), dict(wf=-1), dict(fmt=2),
                dict(off=None), dict(X=None), dict(xs=None), dict(W=None), dict(ws=None), dict(Aq=None), dict(As=None), dict(K=D), dict(Ks=D)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(X=A + 8), dict(W=A + 4), dict(Aq=A + 2), dict(xs=A + 2), dict(ws=A + 1), dict(off=A + 2), dict(As=A + 2),
                dict(K=A + 8, Ks=B), dict(K=A, Ks=B + 2)):
        assert f(**bad) == MISALIGNED, bad


def test_expert_swiglu_backward_refusals(L):  # noqa: F811
    def f(X=A, xs=B, xf=0, W=C, ws=D, wf=0, off=A, K=B, Ks=C, kf=0, R=16, E=4, H=128, I=128, dGU=F, Q=None, Qs=None, fmt=0):
        return L.moe_expert_swiglu_backward(X, xs, xf, W, ws, wf, off, K, Ks, kf, R, E, H, I, dGU, Q, Qs, fmt, None, None)

    assert f(R=0) == OK
    for bad in (dict(E=0), dict(E=257), dict(R=-1), dict(R=2 ** 31 - 1), dict(H=0), dict(H=192), dict(I=0), dict(I=64), dict(I=2 ** 17 + 128),
                dict(xf=2), dict(wf=-1), dict(kf=2), dict(fmt=2), dict(off=None), dict(X=None), dict(xs=None), dict(W=None), dict(ws=None),
                dict(K=None), dict(Ks=None), dict(dGU=None), dict(Q=D), dict(Qs=D)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(X=A + 8), dict(W=A + 4), dict(dGU=A + 2), dict(xs=A + 2), dict(ws=A + 1), dict(off=A + 2), dict(K=A + 8), dict(Ks=A + 2),
                dict(Q=A + 8, Qs=B), dict(Q=A, Qs=B + 2)):
        assert f(**bad) == MISALIGNED, bad


def test_binding_refuses_wrong_shapes():
    x8, xs = torch.zeros((4, 256), dtype=U8), torch.ones((4, 2))
    W, ws, off = torch.zeros((2, 256, 256), dtype=U8), torch.ones((2, 2, 2)), torch.tensor([0, 1, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        moe.expert_swiglu(x8, xs, W, ws, off)
    with pytest.raises(ValueError, match="columns"):
        moe.expert_swiglu(x8[:, :128], xs, W, ws, off)
    with pytest.raises(ValueError, match="multiples of 128"):
        moe.expert_swiglu(x8, xs, W[:, :128], ws, off)
    with pytest.raises(ValueError, match="scale_format"):
        moe.expert_swiglu(x8, xs, W, ws, off, scale_format="e4m3")
    with pytest.raises(ValueError, match="dimensions"):
        moe.expert_swiglu(x8, xs, W[None], ws, off)
    with pytest.raises(TypeError, match="W1_fp8"):
        moe.expert_swiglu(x8, xs, None, ws, off)
    with pytest.raises(ValueError, match="CUDA"):
        moe.expert_swiglu_backward(x8, xs, W, ws, x8, xs, off)
    with pytest.raises(ValueError, match="columns"):
        moe.expert_swiglu_backward(x8, xs, W[:, :128], ws, x8, xs, off)


# ------------------------------------------------------------------ on the GPU

def products(x, W, offs):
    """Each group's rows times its weight [n, red], and the same of magnitudes."""
    y, m = [], []
    for e in range(len(offs) - 1):
        r = x[offs[e]:offs[e + 1]]
        y.append(r @ W[e].T)
        m.append(r.abs() @ W[e].abs().T)
    return torch.cat(y), torch.cat(m)


def check_forward(h, x8, xs, W8, ws, offs, keep=True):
    n, H = offs[-1], x8.shape[1]
    gu, mag = products(ref.decode(x8, xs, 1), ref.decode(W8, ws, ref.BLK), offs)
    s = acc_slack(H, 32, mag)
    if keep:
        assert not ((ref.decode(h.GU_fp8, h.GU_scale, 1)[:n] - gu).abs() > quant_slack(gu, s)).any()
    (g, u), (sg, su) = gu.chunk(2, 1), s.chunk(2, 1)
    a = ref.swiglu(gu)
    # the activation's arithmetic; its slope is at most 1.1
    err = a.abs() * (2.0 ** -21 + g.abs() * 2.0 ** -22) + 1.1 * sg * (u.abs() + su) + (g * torch.sigmoid(g)).abs() * su
    assert not ((ref.decode(h.A_fp8, h.A_scale, 1)[:n] - a).abs() > quant_slack(a, err)).any()


def check_backward(r, dy8, dys, W8, ws, k8, ks, offs):
    n, H = offs[-1], dy8.shape[1]
    da, mag = products(ref.decode(dy8, dys, 1), ref.decode(W8, ws, ref.BLK).transpose(1, 2), offs)
    s, gu = acc_slack(H, 32, mag), ref.decode(k8, ks, 1)[:n]
    g, u = gu.chunk(2, 1)
    want = ref.swiglu_grad(da, gu)
    unit = 2.0 ** -20 + torch.cat([g, g], 1).abs() * 2.0 ** -21
    err = unit * torch.cat([da.abs() * u.abs() * (1 + g.abs()), da.abs() * g.abs()], 1)
    err += ref.swiglu_grad(torch.ones_like(da), gu).abs() * torch.cat([s, s], 1)
    if r.dGU is not None:
        within(r.dGU[:n], want, err)
    if r.dGU_fp8 is not None:
        assert not ((ref.decode(r.dGU_fp8, r.dGU_scale, 1)[:n] - want).abs() > quant_slack(want, err)).any()


def rows(R, C, seed, dev, fmt, std=1.0):  # noqa: F811
    """Rows of very different sizes."""
    by = torch.exp2(torch.randint(-6, 6, (R, 1), generator=torch.Generator().manual_seed(seed + 1000))).to(dev)
    return ref.encode_rows(normal((R, C), seed, dev, std) * by, fmt)


def offsets(counts):
    return [sum(counts[:e]) for e in range(len(counts) + 1)]


SIZES = [  # H, I, formats of the rows, the weights, the results
    (128, 128, "fp32", "fp32", "fp32"),
    (256, 256, "ue8m0", "fp32", "ue8m0"),
    (640, 384, "fp32", "ue8m0", "ue8m0"),    # five blocks of reduction; an odd number of feature blocks
    (1024, 128, "ue8m0", "ue8m0", "fp32"),
    (2176, 640, "fp32", "ue8m0", "fp32"),    # more blocks than the scales are gathered at a time
]


@gpu
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("H,I,xf,wf,fmt", SIZES)
def test_expert_swiglu(dev, counts, H, I, xf, wf, fmt):  # noqa: F811
    E, R, offs = len(counts), sum(counts) + 5, offsets(counts)     # five rows of no group
    x8, xs = rows(R, H, 1, dev, xf)
    W8, ws = ref.encode_weight(normal((E, 2 * I, H), 3, dev, H ** -0.5), wf)
    off, st = ref.offsets_of(counts, dev), status_word(dev)
    out = moe.SwiGLU(*(torch.full((R, c // d), v, dtype=t, device=dev)
                       for c, d, v, t in ((I, 1, 7, U8), (I, 128, 7, U8 if fmt == "ue8m0" else torch.float32),
                                          (2 * I, 1, 7, U8), (2 * I, 128, 7, U8 if fmt == "ue8m0" else torch.float32))))
    h = moe.expert_swiglu(x8, xs, W8, ws, off, scale_format=fmt, out=out, status=st)
    assert st.item() == 0 and h is out
    check_forward(h, x8, xs, W8, ws, offs)
    for t in vars(h).values():
        assert bool((t[offs[-1]:] == 7).all())             # rows of no group are not touched
    alone = moe.expert_swiglu(x8, xs, W8, ws, off, keep=False, scale_format=fmt)
    n = offs[-1]
    assert alone.GU_fp8 is None and torch.equal(alone.A_fp8[:n], h.A_fp8[:n]) and torch.equal(alone.A_scale[:n], h.A_scale[:n])


@gpu
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("H,I,xf,wf,fmt", SIZES)
def test_expert_swiglu_backward(dev, counts, H, I, xf, wf, fmt):  # noqa: F811
    E, R, offs = len(counts), sum(counts) + 5, offsets(counts)
    n, kf = offs[-1], "ue8m0" if fmt == "fp32" else "fp32"
    dy8, dys = rows(R, H, 1, dev, xf)
    k8, ks = rows(R, 2 * I, 2, dev, kf)
    W8, ws = ref.encode_weight(normal((E, H, I), 3, dev, I ** -0.5), wf)
    off, st = ref.offsets_of(counts, dev), status_word(dev)
    out = moe.SwiGLUGrad(torch.full((R, 2 * I), 7, dtype=BF16, device=dev), torch.full((R, 2 * I), 7, dtype=U8, device=dev),
                         torch.full((R, 2 * I // 128), 7, dtype=U8 if fmt == "ue8m0" else torch.float32, device=dev))
    r = moe.expert_swiglu_backward(dy8, dys, W8, ws, k8, ks, off, scale_format=fmt, out=out, status=st)
    assert st.item() == 0 and r is out
    check_backward(r, dy8, dys, W8, ws, k8, ks, offs)
    for t in vars(r).values():
        assert bool((t[n:] == 7).all())
    only = moe.expert_swiglu_backward(dy8, dys, W8, ws, k8, ks, off, fp8=False)
    assert only.dGU_fp8 is None and torch.equal(only.dGU[:n].view(torch.int16), r.dGU[:n].view(torch.int16))
    only = moe.expert_swiglu_backward(dy8, dys, W8, ws, k8, ks, off, bf16=False, scale_format=fmt)
    assert only.dGU is None and torch.equal(only.dGU_fp8[:n], r.dGU_fp8[:n]) and torch.equal(only.dGU_scale[:n], r.dGU_scale[:n])


@gpu
def test_one_group_without_offsets(dev):  # noqa: F811
    H, I, R = 256, 128, 77
    x8, xs = rows(R, H, 5, dev, "fp32")
    W1, s1 = ref.encode_weight(normal((1, 2 * I, H), 6, dev, 0.1), "fp32")
    W2, s2 = ref.encode_weight(normal((1, H, I), 7, dev, 0.1), "fp32")
    h, h2 = moe.expert_swiglu(x8, xs, W1, s1), moe.expert_swiglu(x8, xs, W1[0], s1[0])
    check_forward(h, x8, xs, W1, s1, [0, R])
    assert torch.equal(h.A_fp8, h2.A_fp8) and torch.equal(h.GU_fp8, h2.GU_fp8)
    r = moe.expert_swiglu_backward(x8, xs, W2, s2, h.GU_fp8, h.GU_scale)
    r2 = moe.expert_swiglu_backward(x8, xs, W2[0], s2[0], h.GU_fp8, h.GU_scale)
    check_backward(r, x8, xs, W2, s2, h.GU_fp8, h.GU_scale, [0, R])
    assert torch.equal(r.dGU.view(torch.int16), r2.dGU.view(torch.int16)) and torch.equal(r.dGU_fp8, r2.dGU_fp8)
    empty = moe.expert_swiglu(x8[:0], xs[:0], W1, s1)
    assert empty.A_fp8.shape == (0, I) and empty.GU_scale.shape == (0, 2)
    assert moe.expert_swiglu_backward(x8[:0], xs[:0], W2, s2, h.GU_fp8[:0], h.GU_scale[:0]).dGU.shape == (0, 2 * I)


@gpu
def test_repeated_calls_and_every_position(dev):  # noqa: F811
    """Uneven groups, many tiles: a wait that was missing somewhere would show as a difference; and a row's result
    does not depend on where its group starts or what lies around it."""
    g = torch.Generator().manual_seed(17)
    counts = [int(c) for c in torch.randint(0, 700, (24,), generator=g)]
    R, H, I, offs = sum(counts), 1152, 640, offsets(counts)
    x8, xs = rows(R, H, 18, dev, "ue8m0")
    W1, s1 = ref.encode_weight(normal((24, 2 * I, H), 19, dev, 0.05), "ue8m0")
    W2, s2 = ref.encode_weight(normal((24, H, I), 20, dev, 0.05), "ue8m0")
    off = ref.offsets_of(counts, dev)
    h = moe.expert_swiglu(x8, xs, W1, s1, off)
    r = moe.expert_swiglu_backward(x8, xs, W2, s2, h.GU_fp8, h.GU_scale, off)
    check_forward(h, x8, xs, W1, s1, offs)
    check_backward(r, x8, xs, W2, s2, h.GU_fp8, h.GU_scale, offs)
    for _ in range(30):
        again = moe.expert_swiglu(x8, xs, W1, s1, off)
        assert all(torch.equal(a, b) for a, b in zip(vars(again).values(), vars(h).values()))
        again = moe.expert_swiglu_backward(x8, xs, W2, s2, h.GU_fp8, h.GU_scale, off)
        assert all(torch.equal(a, b) for a, b in zip(vars(again).values(), vars(r).values()))
    for _ in range(30):
        again = moe.expert_swiglu(x8, xs, W1, s1, off, keep=False)
        assert again.GU_fp8 is None and torch.equal(again.A_fp8, h.A_fp8) and torch.equal(again.A_scale, h.A_scale)
    e = max(range(24), key=lambda i: counts[i])
    at = slice(offs[e] + 3, offs[e] + 100)
    part = moe.expert_swiglu(x8[at].contiguous(), xs[at].contiguous(), W1[e], s1[e])
    assert all(torch.equal(a, b[at]) for a, b in zip(vars(part).values(), vars(h).values()))
    part = moe.expert_swiglu_backward(x8[at].contiguous(), xs[at].contiguous(), W2[e], s2[e], h.GU_fp8[at].contiguous(), h.GU_scale[at].contiguous())
    assert all(torch.equal(a, b[at]) for a, b in zip(vars(part).values(), vars(r).values()))


@gpu
@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
def test_scales_need_no_alignment_beyond_their_type(dev, fmt):  # noqa: F811
    counts, H, I = [40, 0, 33], 2048, 256
    x8, xs = rows(73, H, 14, dev, fmt)
    W1, s1 = ref.encode_weight(normal((3, 2 * I, H), 15, dev, 0.05), fmt)
    W2, s2 = ref.encode_weight(normal((3, H, I), 16, dev, 0.05), fmt)
    off = ref.offsets_of(counts, dev)

    def moved(t):
        big = torch.empty(t.numel() + 1, dtype=t.dtype, device=dev)
        big[1:] = t.flatten()
        return big[1:].view(t.shape)

    h = moe.expert_swiglu(x8, xs, W1, s1, off, scale_format=fmt)
    out = moe.SwiGLU(torch.empty_like(h.A_fp8), moved(h.A_scale).zero_(), torch.empty_like(h.GU_fp8), moved(h.GU_scale).zero_())
    moe.expert_swiglu(x8, moved(xs), W1, moved(s1), off, scale_format=fmt, out=out)
    assert all(torch.equal(a, b) for a, b in zip(vars(out).values(), vars(h).values()))
    r = moe.expert_swiglu_backward(x8, xs, W2, s2, h.GU_fp8, h.GU_scale, off, scale_format=fmt)
    out = moe.SwiGLUGrad(torch.empty_like(r.dGU), torch.empty_like(r.dGU_fp8), moved(r.dGU_scale).zero_())
    moe.expert_swiglu_backward(x8, moved(xs), W2, moved(s2), h.GU_fp8, moved(h.GU_scale), off, scale_format=fmt, out=out)
    assert all(torch.equal(a, b) for a, b in zip(vars(out).values(), vars(r).values()))


@gpu
def test_nan_and_infinite_values_keep_to_their_rows(dev):  # noqa: F811
    H, I, R = 256, 256, 70
    x8, xs = ref.encode_rows(normal((R, H), 9, dev), "ue8m0")
    W1, s1 = ref.encode_weight(normal((2, 2 * I, H), 10, dev, 0.1), "ue8m0")
    W2, s2 = ref.encode_weight(normal((2, H, I), 11, dev, 0.1), "ue8m0")
    off = ref.offsets_of([30, 39], dev)
    clean = moe.expert_swiglu(x8, xs, W1, s1, off)
    x8[3, 5] = 0x7F                          # NaN in a row of the first group
    x8[69] = 0x7F                            # the last row of the buffer, in no group
    xs[40] = 255                             # UE8M0's NaN
    xs[20] = 250                             # products that overflow: infinities of both signs
    x8[20] = 0x7E
    h = moe.expert_swiglu(x8, xs, W1, s1, off)
    a, k = ref.decode(h.A_fp8, h.A_scale, 1), ref.decode(h.GU_fp8, h.GU_scale, 1)
    assert bool(a[3].isnan().all() and a[40].isnan().all() and k[3].isnan().all() and k[40].isnan().all())
    assert bool(k[20].isnan().any())         # an infinity is a NaN code under the largest scale
    fine = torch.tensor([i for i in range(69) if i not in (3, 20, 40)], device=dev)
    assert all(torch.equal(x[fine], y[fine]) for x, y in zip(vars(h).values(), vars(clean).values()))
    # a NaN in the checkpoint, in the gradient that comes in
    g8, gs = clean.GU_fp8.clone(), clean.GU_scale.clone()
    y8, ys = ref.encode_rows(normal((R, H), 12, dev), "ue8m0")
    want = moe.expert_swiglu_backward(y8, ys, W2, s2, g8, gs, off)
    g8[7, 300], y8[50, 0], y8[69], g8[69] = 0x7F, 0xFF, 0x7F, 0x7F
    r = moe.expert_swiglu_backward(y8, ys, W2, s2, g8, gs, off)
    # column 300 is of the up half: dg = da u s (1 + g (1 - s)) has it, du = da g s does not
    assert r.dGU[7].isnan().nonzero().flatten().tolist() == [300 - I]
    assert bool(r.dGU[50].isnan().all()) and bool(ref.decode(r.dGU_fp8, r.dGU_scale, 1)[50].isnan().all())
    q = ref.decode(r.dGU_fp8, r.dGU_scale, 1)[7]
    assert q.isnan().nonzero().flatten().tolist() == [300 - I]
    fine = torch.tensor([i for i in range(69) if i not in (7, 50)], device=dev)
    assert all(torch.equal(x[fine], y[fine]) for x, y in zip(vars(r).values(), vars(want).values()))
    g8[8, 20] = 0x7F                         # of the gate half: both have it
    r = moe.expert_swiglu_backward(y8, ys, W2, s2, g8, gs, off)
    assert r.dGU[8].isnan().nonzero().flatten().tolist() == [20, 20 + I]


@gpu
def test_bad_scales_and_offsets_are_reported(dev):  # noqa: F811
    R, n = 40, 128
    x8, xs = ref.encode_rows(normal((R, n), 11, dev), "fp32")
    W1, s1 = ref.encode_weight(normal((2, 2 * n, n), 12, dev), "fp32")
    W2, s2 = ref.encode_weight(normal((2, n, n), 13, dev), "fp32")
    k8, ks = ref.encode_rows(normal((R, 2 * n), 14, dev), "fp32")
    good = ref.offsets_of([20, 20], dev)

    def status(call, *args):
        st = status_word(dev)
        call(*args, status=st)
        return st.item()

    for poison in (3.0, -1.0, 0.0, float("inf"), float("nan")):
        bad, bad_k = xs.clone(), ks.clone()
        bad[7], bad_k[9, 1] = poison, poison
        assert status(moe.expert_swiglu, x8, bad, W1, s1, good) == moe.ERR_BAD_SCALE, poison
        assert status(moe.expert_swiglu_backward, x8, bad, W2, s2, k8, ks, good) == moe.ERR_BAD_SCALE, poison
        assert status(moe.expert_swiglu_backward, x8, xs, W2, s2, k8, bad_k, good) == moe.ERR_BAD_SCALE, poison
    assert status(moe.expert_swiglu, x8, xs, W1, torch.full_like(s1, 3.0), good) == moe.ERR_BAD_SCALE
    for off in ([0, 20, 41], [-1, 20, 40], [0, 30, 20], [50, 60, 70]):
        o, st = torch.tensor(off, dtype=torch.int32, device=dev), status_word(dev)
        out = torch.full((R, 2 * n), 7.0, dtype=BF16, device=dev)
        assert status(moe.expert_swiglu, x8, xs, W1, s1, o) == moe.ERR_BAD_INDEX, off
        moe.expert_swiglu_backward(x8, xs, W2, s2, k8, ks, o, out=moe.SwiGLUGrad(out, None, None), status=st)
        assert st.item() == moe.ERR_BAD_INDEX, off
    assert bool((out == 7.0).all())          # [50, 60, 70]: both groups outside


@gpu
def test_offsets_beyond_32_bits(dev):  # noqa: F811
    """2^31 bytes of checkpoint and more: the last rows."""
    H, I, R, last = 128, 1024, (1 << 20) + 77, 300
    x8, xs = ref.encode_rows(normal((last, H), 31, dev), "ue8m0")
    W1, s1 = ref.encode_weight(normal((2, 2 * I, H), 32, dev, 0.1), "ue8m0")
    W2, s2 = ref.encode_weight(normal((2, H, I), 33, dev, 0.1), "ue8m0")
    X8 = torch.zeros((R, H), dtype=U8, device=dev)
    Xs = torch.full((R, 1), 127, dtype=U8, device=dev)
    X8[-last:], Xs[-last:] = x8, xs
    off = torch.tensor([0, R - 100, R], dtype=torch.int32, device=dev)
    h = moe.expert_swiglu(X8, Xs, W1, s1, off, scale_format="ue8m0")
    ends = torch.tensor([0, last - 100, last], dtype=torch.int32, device=dev)
    want = moe.expert_swiglu(x8, xs, W1, s1, ends, scale_format="ue8m0")
    assert all(torch.equal(a[-last:], b) for a, b in zip(vars(h).values(), vars(want).values()))
    r = moe.expert_swiglu_backward(X8, Xs, W2, s2, h.GU_fp8, h.GU_scale, off, scale_format="ue8m0")
    want = moe.expert_swiglu_backward(x8, xs, W2, s2, want.GU_fp8, want.GU_scale, ends, scale_format="ue8m0")
    assert all(torch.equal(a[-last:], b) for a, b in zip(vars(r).values(), vars(want).values()))
    assert not h.A_fp8[:-last].any() and not r.dGU[:-last].any()


@gpu
def test_agrees_with_the_calls_it_joins(dev):  # noqa: F811
    """Against expert_gemm, swiglu and their gradients, whose bf16 rows between are the only difference: a half step
    of bf16 (2^-8) ahead of the activation, half a step of E4M3 (2^-4) on each side."""
    counts, H, I = [130, 0, 61, 300], 512, 256
    R, off = sum(counts), ref.offsets_of(counts, dev)
    x8, xs = rows(R, H, 41, dev, "fp32")
    W1, s1 = ref.encode_weight(normal((4, 2 * I, H), 42, dev, H ** -0.5), "fp32")
    W2, s2 = ref.encode_weight(normal((4, H, I), 43, dev, I ** -0.5), "fp32")
    h = moe.expert_swiglu(x8, xs, W1, s1, off)
    g = moe.swiglu(moe.expert_gemm(x8, xs, W1, s1, off))
    for a, b, c, d in ((h.A_fp8, h.A_scale, g.A_fp8, g.A_scale), (h.GU_fp8, h.GU_scale, g.GU_fp8, g.GU_scale)):
        u, v = ref.decode(a, b, 1), ref.decode(c, d, 1)
        assert (u - v).norm() <= 2.0 ** -4 * v.norm()
    r = moe.expert_swiglu_backward(x8, xs, W2, s2, h.GU_fp8, h.GU_scale, off)
    b = moe.swiglu_backward(moe.expert_gemm(x8, xs, W2, s2, off, transpose=True), h.GU_fp8, h.GU_scale)
    assert (r.dGU.double() - b.dGU.double()).norm() <= 3 * 2.0 ** -8 * b.dGU.double().norm()
    u, v = ref.decode(r.dGU_fp8, r.dGU_scale, 1), ref.decode(b.dGU_fp8, b.dGU_scale, 1)
    assert (u - v).norm() <= 2.0 ** -4 * v.norm()


@gpu
def test_captured_and_on_another_stream(dev):  # noqa: F811
    counts, H, I = [33, 0, 70], 256, 128
    R, off = sum(counts), ref.offsets_of(counts, dev)
    x8, xs = rows(R, H, 51, dev, "ue8m0")
    W1, s1 = ref.encode_weight(normal((3, 2 * I, H), 52, dev, 0.1), "ue8m0")
    W2, s2 = ref.encode_weight(normal((3, H, I), 53, dev, 0.1), "ue8m0")
    h = moe.expert_swiglu(x8, xs, W1, s1, off)
    r = moe.expert_swiglu_backward(x8, xs, W2, s2, h.GU_fp8, h.GU_scale, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h2 = moe.expert_swiglu(x8, xs, W1, s1, off, stream=side)
    r2 = moe.expert_swiglu_backward(x8, xs, W2, s2, h2.GU_fp8, h2.GU_scale, off, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3 = moe.expert_swiglu(x8, xs, W1, s1, off)
        r3 = moe.expert_swiglu_backward(x8, xs, W2, s2, h3.GU_fp8, h3.GU_scale, off)
    for _ in range(3):
        for t in (*vars(h3).values(), *vars(r3).values()):
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for got in (h2, h3):
        assert all(torch.equal(a, b) for a, b in zip(vars(got).values(), vars(h).values()))
    for got in (r2, r3):
        assert all(torch.equal(a, b) for a, b in zip(vars(got).values(), vars(r).values()))
