"""Rows out of the ordinary in the norm's gradient: zeros, rows whose squares leave 32 bits (rstd 0), infinities and NaN.  What
a row of the first two kinds gives is the formula's; the last two reach their own row and the weight's gradient; the other
rows' gradients stay what they are, to the bit."""
import pytest
import torch

import combine_moe_route_02_gb300 as moe
from test_experts import dev, gpu, normal  # noqa: F401
from test_norms import BF16, F32, U, weight

N, AT = 300, (1, 7, 299)


def run(x, dy, w, ds, dev):  # noqa: F811
    n = moe.rms_norm(x, w)
    return n, moe.rms_norm_backward(dy, n.S, w, n.rstd, dS=ds)


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@gpu
@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("H", [256, 1184, 2048, 8200])
@pytest.mark.parametrize("kind", ["zero", "tiny", "beyond", "infinite", "nan"])
def test_special_rows_of_the_gradient(dev, kind, H, stream):  # noqa: F811
    x, dy, w = normal((N, H), 1, dev), normal((N, H), 2, dev), weight(H, F32, dev)
    ds = normal((N, H), 3, dev) if stream else None
    _, clean = run(x.clone(), dy, w, ds, dev)
    at = torch.tensor(AT, device=dev)
    if kind in ("infinite", "nan"):
        x[at, 5] = float(kind.replace("infinite", "-inf"))
    else:
        x[at] = {"zero": torch.zeros_like, "tiny": lambda t: t * 2.0 ** -100, "beyond": lambda t: t * 2.0 ** 100}[kind](x[at])
    if kind == "beyond":
        dy[at] *= 2.0 ** 40          # dy s is beyond 32 bits, dy (s rstd) is 0
    n, g = run(x, dy, w, ds, dev)
    rest = torch.ones(N, dtype=torch.bool, device=dev)
    rest[at] = False
    assert same(g.dX[rest], clean.dX[rest])
    if kind == "nan":
        assert bool(g.dX[at].isnan().all()) and bool(g.dweight.isnan().all())
        return
    r = n.rstd.double()[:, None]
    xh = x.double() * r
    terms = dy.double() * xh         # (infinity times 0 is the formula's NaN)
    dw, mag = terms.sum(0), terms.abs().sum(0)
    if kind == "infinite":
        assert not n.rstd[at].any() and bool(g.dX[at].isnan().all())
        assert g.dweight.isnan().nonzero().flatten().tolist() == [5] == dw.isnan().nonzero().flatten().tolist()
        dw[5] = mag[5] = g.dweight[5] = 0
    else:
        assert kind != "beyond" or not n.rstd[at].any()
        assert n.rstd[at].allclose(torch.tensor(0.0 if kind == "beyond" else 1000.0, device=dev), rtol=2.0 ** -18, atol=0)
        d = dy.double() * w.double()
        mean, size = (d * xh).mean(1, keepdim=True), (d * xh).abs().mean(1, keepdim=True)
        want = r * (d - xh * mean) + (ds.double() if stream else 0)
        slack = r * (xh.abs() * 64 * U * size + 4 * U * (d.abs() + (xh * mean).abs())) + 2 * U * want.abs()
        assert not ((g.dX.double() - want).abs() > slack + 2.0 ** -8 * (want.abs() + slack)).any()
        if kind == "beyond":         # nothing but the stream's gradient comes through such a row
            assert same(g.dX[at], ds[at]) if stream else not g.dX[at].any()
    # a row's term rounded twice; 300 rows are at most 64 in a thread, four warps', and the table's 300 by 8, 3, 2 and 32 steps
    assert not ((g.dweight.double() - dw).abs() > (64 + 4 + 8 + 3 + 2 + 32 + 2) * U * mag).any()
