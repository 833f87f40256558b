"""The norms around the experts against their formulas in 64 bits: the RMS norm with the residual's addition and its
gradient, the norm of all gradients and the clipping.

Tolerances.  A sum of n positive terms in 32 bits is off by at most its depth times 2^-24 of itself.  A row's sum is
32 squares in a thread, 5 steps of a warp and 16 warps at the most, a root halves that, and a division, a root and
two products follow: 40 * 2^-24 < 2^-18 for rstd and y.
"""
import ctypes
import math

import pytest
import torch

import combine_moe_route_02_gb300 as moe
import experts_ref as ref
from test_experts import A, B, C, D, F, INVALID, MISALIGNED, OK, WORKSPACE, L, dev, gpu, normal, quant_slack, within  # noqa: F401

BF16, U8, F32 = torch.bfloat16, torch.uint8, torch.float32
U = 2.0 ** -24


# ------------------------------------------------------------------ on the CPU: refusals

def test_rms_norm_refusals(L):  # noqa: F811
    def f(X=A, res=None, w=B, wt=0, eps=1e-6, N=4, H=256, S=None, Y=C, Q=None, Qs=None, fmt=0, rstd=D):
        return L.moe_rms_norm(X, res, w, wt, eps, N, H, S, Y, Q, Qs, fmt, rstd, None)

    assert f(N=0) == OK
    for bad in (dict(X=None), dict(w=None), dict(wt=2), dict(wt=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=2.0), dict(eps=math.nan), dict(N=-1),
                dict(N=2 ** 31), dict(H=0), dict(H=12), dict(H=16392), dict(Y=None), dict(Q=F), dict(Qs=F), dict(Q=F, Qs=A, H=264), dict(fmt=2),
                dict(res=F), dict(S=F)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(X=A + 2), dict(w=B + 4), dict(Y=C + 8), dict(res=F + 2, S=A), dict(res=F, S=A + 8), dict(Q=F + 8, Qs=A), dict(Q=F, Qs=A + 2), dict(rstd=D + 2)):
        assert f(**bad) == MISALIGNED, bad


def test_rms_norm_backward_refusals(L):  # noqa: F811
    need = L.moe_rms_norm_backward_workspace_size(4, 256)
    assert need > 0 and L.moe_rms_norm_backward_workspace_size(4, 12) == 0 and L.moe_rms_norm_backward_workspace_size(-1, 256) == 0

    def f(dY=A, S=B, w=C, wt=0, r=D, dS=None, add=None, N=4, H=256, dX=F, dw=A, st=None, ws=B, n=need):
        return L.moe_rms_norm_backward(dY, S, w, wt, r, dS, add, N, H, dX, dw, st, ws, n, None)

    for bad in (dict(dY=None), dict(S=None), dict(w=None), dict(r=None), dict(dX=None), dict(dw=None), dict(wt=2), dict(N=-1), dict(N=2 ** 31),
                dict(H=0), dict(H=12), dict(H=16392), dict(dw=None, N=0)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(dY=A + 2), dict(S=B + 8), dict(w=C + 2), dict(r=D + 2), dict(dS=A + 2), dict(add=A + 2), dict(dX=F + 8), dict(dw=A + 2), dict(st=A + 2), dict(ws=B + 4)):
        assert f(**bad) == MISALIGNED, bad
    assert f(ws=None) == WORKSPACE and f(n=need - 1) == WORKSPACE


def test_clip_refusals(L):  # noqa: F811
    need = L.moe_grad_norm_workspace_size(2)
    assert need > 0 and L.moe_grad_norm_workspace_size(-1) == 0 and L.moe_grad_norm_workspace_size(2000) == 2 * need

    def f(src=(A, B), dst=(C, D), sizes=(5, 7), types=(0, 1), n=2, most=1.0, norm=F, ws=A, nb=need, clip=True):
        P, I64, I32 = ctypes.c_void_p * 2, ctypes.c_int64 * 2, ctypes.c_int * 2
        s, d = src and P(*src), dst and P(*dst)
        k, t = sizes and I64(*sizes), types and I32(*types)
        if clip:
            return L.moe_clip_grad_norm(s, d, k, t, n, most, norm, ws, nb, None)
        return L.moe_grad_norm(s, k, t, n, norm, ws, nb, None)

    for bad in (dict(src=None), dict(sizes=None), dict(types=None), dict(n=-1), dict(sizes=(-1, 7)), dict(sizes=(2 ** 42, 1)), dict(sizes=(2 ** 62, 2 ** 62)),
                dict(types=(0, 2)), dict(src=(A, None)), dict(norm=None)):
        assert f(**bad) == INVALID, bad
        assert f(clip=False, **bad) == INVALID, bad
    for bad in (dict(dst=(C, None)), dict(most=-1.0), dict(most=math.nan)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(src=(A + 2, B)), dict(src=(A, B + 1)), dict(dst=(C + 2, D)), dict(dst=(C, D + 1)), dict(norm=F + 2), dict(ws=A + 8)):
        assert f(**bad) == MISALIGNED, bad
    assert f(ws=None) == WORKSPACE and f(nb=need - 1) == WORKSPACE


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x, w = torch.zeros((4, 256), dtype=BF16), torch.ones(256)
    with pytest.raises(ValueError, match="CUDA"):
        moe.rms_norm(x, w)
    with pytest.raises(ValueError, match="dimensions"):
        moe.rms_norm(x[0], w)
    with pytest.raises(ValueError, match="scale_format"):
        moe.rms_norm(x, w, scale_format="e4m3")
    with pytest.raises(ValueError, match="CUDA"):
        moe.rms_norm_backward(x, x, w, torch.ones(4))
    with pytest.raises(ValueError, match="CUDA"):
        moe.grad_norm([w])
    with pytest.raises(TypeError, match="list"):
        moe.grad_norm([1.0])
    with pytest.raises(ValueError, match="max_norm"):
        moe.clip_grad_norm([w], -1.0)


# ------------------------------------------------------------------ the RMS norm

SHAPES = [(1, 8), (1, 128), (3, 256), (5, 264), (17, 1024), (33, 1032), (7, 2048), (130, 2056), (9, 4096), (4, 4104), (3, 8192), (2, 8200),
          (3, 16384), (1000, 128), (701, 640)]


def stream_rows(N, H, seed, dev):  # noqa: F811
    """Rows of very different lengths, with one column far larger than the rest."""
    x = normal((N, H), seed, dev).float() * torch.exp2(torch.randint(-8, 8, (N, 1), generator=torch.Generator().manual_seed(seed)).float()).to(dev)
    x[:, H // 3] *= 50
    return x.to(BF16)


def weight(H, dtype, dev):  # noqa: F811
    return (1 + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(H))).to(dtype).to(dev)


@gpu
@pytest.mark.parametrize("N,H", SHAPES)
@pytest.mark.parametrize("residual,wt,fmt", [(False, F32, "fp32"), (True, BF16, "ue8m0"), (True, F32, "fp32")])
def test_rms_norm(dev, N, H, residual, wt, fmt):  # noqa: F811
    x, w = stream_rows(N, H, 1, dev), weight(H, wt, dev)
    res = stream_rows(N, H, 2, dev) if residual else None
    fp8 = H % 128 == 0
    r = moe.rms_norm(x, w, residual=res, eps=1e-5, fp8=fp8, scale_format=fmt)
    s = x.double() + (res.double() if residual else 0)
    if residual:
        assert torch.equal(r.S.view(torch.int16), s.to(BF16).view(torch.int16))
        s = r.S.double()
    else:
        assert r.S is x
    rstd = (s.square().mean(1) + 1e-5).rsqrt()
    y = s * rstd[:, None] * w.double()
    assert not ((r.rstd.double() - rstd).abs() > 2.0 ** -18 * rstd).any()
    within(r.Y, y, 2.0 ** -18 * y.abs())
    if fp8:
        assert not ((ref.decode(r.Y_fp8, r.Y_scale, 1) - y).abs() > quant_slack(y, 2.0 ** -18 * y.abs())).any()
        only = moe.rms_norm(x, w, residual=res, eps=1e-5, bf16=False, fp8=True, scale_format=fmt)
        assert only.Y is None and torch.equal(only.Y_fp8, r.Y_fp8) and torch.equal(only.Y_scale, r.Y_scale)
    # in place: the stream over the residual, y over x
    x2, res2 = x.clone(), res.clone() if residual else None
    out = moe.RMSNorm(x2, None, None, res2 if residual else x2, None)
    moe.rms_norm(x2, w, residual=res2, eps=1e-5, out=out)
    assert torch.equal(x2.view(torch.int16), r.Y.view(torch.int16))
    if residual:
        assert torch.equal(res2.view(torch.int16), r.S.view(torch.int16))


@gpu
def test_rms_norm_special_rows(dev):  # noqa: F811
    x, w = normal((8, 256), 3, dev), weight(256, F32, dev)
    clean = moe.rms_norm(x, w, fp8=True)
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 200] = float("inf")
    x[4] = 1e-30
    r = moe.rms_norm(x, w, fp8=True)
    assert bool((r.Y[1] == 0).all()) and bool((ref.decode(r.Y_fp8, r.Y_scale, 1)[1] == 0).all()) and abs(float(r.rstd[1]) - 1000) <= 1e-3
    assert bool(r.Y[2].isnan().all())
    assert r.Y[3].isnan().nonzero().flatten().tolist() == [200] and float(r.rstd[3]) == 0   # (infinity times 0)
    within(r.Y[4], x[4].double() * 1000 * w.double(), 2.0 ** -18 * 1e-27)
    for i in (0, 5, 6, 7):
        assert torch.equal(r.Y[i], clean.Y[i]) and torch.equal(r.Y_fp8[i], clean.Y_fp8[i]) and r.rstd[i] == clean.rstd[i]


@gpu
def test_no_rows(dev):  # noqa: F811
    w, add = weight(256, F32, dev), torch.randn(256).to(dev)
    x = torch.empty((0, 256), dtype=BF16, device=dev)
    assert moe.rms_norm(x, w, residual=x, fp8=True).Y.shape == (0, 256)
    g = moe.rms_norm_backward(x, x, w, torch.empty(0, device=dev), add=add)
    assert g.dX.shape == (0, 256) and torch.equal(g.dweight, add)
    assert not moe.rms_norm_backward(x, x, w, torch.empty(0, device=dev)).dweight.any()


@gpu
@pytest.mark.parametrize("N,H", SHAPES + [(5000, 512), (2500, 4096)])
@pytest.mark.parametrize("stream,add,wt", [(False, True, F32), (True, False, BF16)])
def test_rms_norm_backward(dev, N, H, stream, add, wt):  # noqa: F811
    s, w, dy = stream_rows(N, H, 1, dev), weight(H, wt, dev), normal((N, H), 4, dev)
    ds = normal((N, H), 5, dev, 0.3) if stream else None
    base = torch.randn(H, generator=torch.Generator().manual_seed(6)).to(dev) if add else None
    rstd = (s.double().square().mean(1) + 1e-6).rsqrt().float()
    g = moe.rms_norm_backward(dy, s, w, rstd, dS=ds, add=base)
    r = rstd.double()[:, None]
    xh, d = s.double() * r, dy.double() * w.double()
    mean, size = (d * xh).mean(1, keepdim=True), (d * xh).abs().mean(1, keepdim=True)
    want = r * (d - xh * mean)
    # the row's sum; the factor of s (three products and a division, of which two are the mean's own and in its 64),
    # d's product, s's and dS's sum and the whole, each rounded once; where dS is larger than the whole it is at most
    # the whole and the two terms
    slack = r * (xh.abs() * 64 * U * size + 4 * U * (d.abs() + (xh * mean).abs()))
    if stream:
        want = want + ds.double()
        slack = slack + 2 * U * want.abs()
    within(g.dX, want, slack)
    # 64 rows at a time, those sums (a CTA has at least N / 608 rows where it has more than one), four rows of a warp's
    # CTA, then the table's rows (at most 1216) as 32 x 8 sums
    each = N / 608
    depth = min(each + 1, 64) + each / 64 + 4 + 1216 / 256 + 3 + 32 + 2
    dw, mag = (dy.double() * xh).sum(0), (dy.double() * xh).abs().sum(0)
    if add:
        dw, mag = dw + base.double(), mag + base.double().abs()
    assert not ((g.dweight.double() - dw).abs() > depth * U * mag + 2 * U * mag).any()
    for _ in range(3):
        again = moe.rms_norm_backward(dy, s, w, rstd, dS=ds, add=base)
        assert torch.equal(again.dX.view(torch.int16), g.dX.view(torch.int16)) and torch.equal(again.dweight, g.dweight)
    # in place: dX over dY, or over what it adds; the weight's gradient over what it is added to
    buf, acc = (ds if stream else dy).clone(), base.clone() if add else torch.empty(H, device=dev)
    moe.rms_norm_backward(dy if stream else buf, s, w, rstd, dS=buf if stream else None, add=acc if add else None, out=moe.RMSNormGrad(buf, acc))
    assert torch.equal(buf.view(torch.int16), g.dX.view(torch.int16)) and torch.equal(acc, g.dweight)


@gpu
def test_rms_norm_gradient_against_differences(dev):  # noqa: F811
    """The formula that the kernel is held to, against differences of the norm in 64 bits."""
    g = torch.Generator().manual_seed(8)
    s, w, dy = (torch.randn(n, generator=g, dtype=torch.float64) for n in ((3, 16), (16,), (3, 16)))

    def f(s, w):
        return (dy * s * (s.square().mean(1, keepdim=True) + 1e-3).rsqrt() * w).sum()

    r = (s.square().mean(1, keepdim=True) + 1e-3).rsqrt()
    xh, d, h = s * r, dy * w, 1e-6
    dx, dw = r * (d - xh * (d * xh).mean(1, keepdim=True)), (dy * xh).sum(0)
    for i in range(3):
        for j in range(16):
            e = torch.zeros_like(s)
            e[i, j] = h
            assert abs(float((f(s + e, w) - f(s - e, w)) / (2 * h) - dx[i, j])) < 1e-8
    for j in range(16):
        e = torch.zeros_like(w)
        e[j] = h
        assert abs(float((f(s, w + e) - f(s, w - e)) / (2 * h) - dw[j])) < 1e-8


@gpu
def test_rms_norm_of_integers_is_exact(dev):  # noqa: F811
    """Rows of +-1 and weights that are powers of two: the gradient in whole numbers, to the last bit."""
    g = torch.Generator().manual_seed(9)
    s = (torch.randint(0, 2, (300, 512), generator=g) * 2 - 1).to(BF16).to(dev)
    dy = torch.randint(-4, 5, (300, 512), generator=g).to(BF16).to(dev)
    w = torch.exp2(torch.randint(-2, 3, (512,), generator=g).float()).to(dev)
    ones = torch.ones(300, device=dev)
    got = moe.rms_norm_backward(dy, s, w, ones)
    assert torch.equal(got.dweight.double(), (dy.double() * s.double()).sum(0))
    d = dy.double() * w.double()
    assert torch.equal(got.dX, (d - s.double() * (d * s.double()).mean(1, keepdim=True)).to(BF16))


@gpu
def test_rows_beyond_32_bits(dev):  # noqa: F811
    N, H, last = 270000, 8192, 40       # 2.2e9 elements
    x = torch.zeros((N, H), dtype=BF16, device=dev)
    x[-last:], w = normal((last, H), 11, dev), weight(H, F32, dev)
    r = moe.rms_norm(x, w, fp8=True, scale_format="ue8m0")
    want = moe.rms_norm(x[-last:].clone(), w, fp8=True, scale_format="ue8m0")
    assert torch.equal(r.Y[-last:], want.Y) and torch.equal(r.Y_fp8[-last:], want.Y_fp8) and torch.equal(r.Y_scale[-last:], want.Y_scale)
    assert torch.equal(r.rstd[-last:], want.rstd) and not r.Y[:-last].any()
    g = moe.rms_norm_backward(x, x, w, r.rstd)
    part = moe.rms_norm_backward(x[-last:].clone(), x[-last:].clone(), w, want.rstd)
    assert torch.equal(g.dX[-last:], part.dX) and not g.dX[:-last].any()
    xh = x[-last:].double() * want.rstd.double()[:, None]
    terms = x[-last:].double() * xh
    assert not ((g.dweight.double() - terms.sum(0)).abs() > 120 * U * terms.abs().sum(0)).any()


# ------------------------------------------------------------------ the norm of all gradients

def tensors(sizes, dtypes, seed, dev, std=1.0):  # noqa: F811
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(t).to(dev) for n, t in zip(sizes, dtypes)]


def exact_norm(grads):
    return math.sqrt(sum(float(t.double().square().sum()) for t in grads))


# 65 squares of a thread in 32 bits, halved by the root, the root's own rounding: 34 * 2^-24
NORM_TOL = 34 * U


def check_clip(grads, most, **k):
    norm = exact_norm(grads)
    before = [t.clone() for t in grads]
    got = moe.clip_grad_norm(grads, most, **k)
    assert got.dtype == F32 and got.shape == (1,) and abs(float(got) - norm) <= NORM_TOL * norm + 1e-45
    c = min(1.0, most / (norm + 1e-6))
    for b, t in zip(before, k.get("out") or grads):
        # the coefficient's error is the norm's and two roundings
        within(t, b.double() * c, (NORM_TOL + 2 * U) * b.double().abs() * c if c < 1 else 0 * b.double())
    if k.get("out"):
        assert all(torch.equal(a, b) for a, b in zip(before, grads))


@gpu
@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [7, 8, 9], [16384, 16385, 16383, 8192, 8193, 3], [100003, 1, 250000], [3] * 128, [5] * 129, [0] * 3])
@pytest.mark.parametrize("types", [(F32,), (BF16,), (F32, BF16)])
def test_clip(dev, sizes, types):  # noqa: F811
    dtypes = [types[i % len(types)] for i in range(len(sizes))]
    for bound in (0.25, 4.0):
        grads = tensors(sizes, dtypes, len(sizes), dev)
        norm = exact_norm(grads)
        assert abs(float(moe.grad_norm(grads)) - norm) <= NORM_TOL * norm
        check_clip([t.clone() for t in grads], bound * (norm + 1e-6))
        check_clip(grads, bound * (norm + 1e-6), out=[torch.empty_like(t) for t in grads])
        check_clip(grads, 0.0, out=[torch.empty_like(t) for t in grads])
    assert float(moe.grad_norm([])) == 0 and float(moe.clip_grad_norm([], 1.0)) == 0


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_clip_any_alignment(dev, dtype):  # noqa: F811
    """Every shift of the input against every shift of the output; what lies around the tensors stays."""
    n, per = 40000, 16 // dtype.itemsize
    src = tensors([n + per], [dtype], 1, dev)[0]
    for a in range(per):
        for b in range(per):
            x, buf = src[a:a + n], torch.full((n + 2 * per,), 7, dtype=dtype, device=dev)
            y = buf[b:b + n]
            check_clip([x], 10.0, out=[y])
            assert bool((buf[:b] == 7).all()) and bool((buf[b + n:] == 7).all())
        y = src.clone()
        check_clip([y[a:a + n]], 10.0)
        assert torch.equal(y[:a], src[:a]) and torch.equal(y[a + n:], src[a + n:])
        for short in (1, 2, per - 1, per + 1):
            check_clip([src.clone()[a:a + short]], 0.01)


@gpu
def test_clip_many_tensors(dev):  # noqa: F811
    """More than one launch takes: 2500 tensors, views of one buffer."""
    g = torch.Generator().manual_seed(3)
    sizes = [int(n) for n in torch.randint(0, 400, (2500,), generator=g)]
    flat = torch.randn(sum(sizes), generator=g).to(dev)
    for out in (None, torch.empty_like(flat)):
        buf = flat.clone()
        grads = list(buf.split(sizes))
        norm = exact_norm([flat])
        check_clip(grads, norm / 3, **({} if out is None else {"out": list(out.split(sizes))}))


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [1e30, 3e37, 1e-25, 1e-38])
def test_norm_beyond_the_range_of_squares(dev, dtype, size):  # noqa: F811
    grads = [t * size for t in tensors([70000, 33], [dtype, F32], 5, dev, 0.5)]
    norm = exact_norm(grads)
    if norm < 3.4e38:
        assert abs(float(moe.grad_norm(grads)) - norm) <= NORM_TOL * norm + 2.0 ** -149
    mixed = grads + tensors([5000], [F32], 6, dev)
    norm = exact_norm(mixed)
    if norm < 3.4e38:
        assert abs(float(moe.grad_norm(mixed)) - norm) <= NORM_TOL * norm


@gpu
@pytest.mark.parametrize("poison", [float("inf"), float("-inf"), float("nan")])
def test_a_norm_that_is_not_finite_leaves_the_tensors(dev, poison):  # noqa: F811
    for dtype in (F32, BF16):
        grads = tensors([20000, 3], [dtype, F32], 7, dev)
        grads[0][12345] = poison
        before = [t.clone() for t in grads]
        out = [torch.zeros_like(t) for t in grads]
        for k in ({}, {"out": out}):
            norm = float(moe.clip_grad_norm(grads, 1e-3, **k))
            assert math.isnan(norm) if math.isnan(poison) else norm == math.inf
        for a, b, c in zip(grads, before, out):
            assert torch.equal(a.nan_to_num(5.0), b.nan_to_num(5.0)) and torch.equal(c.nan_to_num(5.0), b.nan_to_num(5.0))


@gpu
def test_clip_refuses_a_tensor_listed_twice_and_unlike_outputs(dev):  # noqa: F811
    a, b = tensors([100, 200], [F32, F32], 8, dev)
    with pytest.raises(ValueError, match="twice"):
        moe.clip_grad_norm([a, b, a], 1.0)
    with pytest.raises(ValueError, match="twice"):
        moe.clip_grad_norm([a, a], 1.0, out=[b[:100], b[:100]])
    assert abs(float(moe.grad_norm([a, a])) - math.sqrt(2) * exact_norm([a])) <= 2 * NORM_TOL * exact_norm([a])
    with pytest.raises(ValueError, match="sizes and types"):
        moe.clip_grad_norm([a], 1.0, out=[b])
    with pytest.raises(ValueError, match="sizes and types"):
        moe.clip_grad_norm([a, b], 1.0, out=[a])
    with pytest.raises(TypeError, match=r"grads\[1\]"):
        moe.grad_norm([a, b.half()])
    with pytest.raises(ValueError, match="contiguous"):
        moe.grad_norm([a, b.view(20, 10).T])
    with pytest.raises(ValueError, match="CUDA"):
        moe.grad_norm([a, b.cpu()])


@gpu
def test_a_tensor_beyond_32_bits(dev):  # noqa: F811
    n = (1 << 31) + 12345
    x = torch.zeros(n, dtype=BF16, device=dev)
    x[-3:], x[5] = 2.0, 1.0
    assert float(moe.grad_norm([x])) == float(torch.tensor(13.0).sqrt())
    moe.clip_grad_norm([x], 0.5 * math.sqrt(13) + 5e-7)
    assert x[-3:].tolist() == [1.0] * 3 and float(x[5]) == 0.5 and int(x.count_nonzero()) == 4


@gpu
def test_norms_captured_and_on_another_stream(dev):  # noqa: F811
    x, res, w = stream_rows(50, 640, 1, dev), stream_rows(50, 640, 2, dev), weight(640, F32, dev)
    grads = tensors([3000, 41], [F32, BF16], 9, dev)

    def step(**k):
        r = moe.rms_norm(x, w, residual=res, fp8=True, **k)
        g = moe.rms_norm_backward(x, r.S, w, r.rstd, dS=res, **k)
        out = [torch.zeros_like(t) for t in grads]
        return [r.Y, r.Y_fp8, r.Y_scale, r.S, r.rstd, g.dX, g.dweight, moe.clip_grad_norm(grads, 1.0, out=out, **k), moe.grad_norm(grads, **k), *out]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = step(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[:9], want[:9]))
    graphs = []
    for _ in range(2):                   # two graphs alive at once, replayed in turn with plain calls between
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        graphs.append((graph, got))
    for _ in range(3):
        for graph, got in graphs:
            for t in got:
                t.zero_()
            graph.replay()
            plain = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip(plain, want))
