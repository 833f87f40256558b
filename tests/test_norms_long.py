"""The norm's gradient where a CTA adds to its row of the table more than once (every 64 groups of rows), and at the widest
rows of a warp and the narrowest of several.

Tolerance of the weight's gradient, in steps of 2^-24 of the terms' magnitudes: 64 rows are summed one after the other in
a thread; those sums, from each of four warps where a row is a warp's, in the table: 4 for each 64 groups of a CTA; the
table's rows (1216 at the most) two at a time in each of eight sums, these by 3 steps, two more across lanes, 32 one after
the other, and what is added; two roundings of the term itself (s * rstd, its product with dy inside the sum's).
"""
import pytest
import torch

import combine_moe_route_02_gb300 as moe
from test_experts import dev, gpu, normal  # noqa: F401
from test_norms import BF16, F32, U, stream_rows, weight

# rows, columns, groups of a CTA (its rows, or fours of them): the CTAs are six or four an SM, or as many as the threads allow
CASES = [(600001, 128, 165), (400003, 1184, 165), (150001, 1192, 124), (100003, 4096, 165), (20003, 8200, 132), (25001, 16384, 165)]


@gpu
@pytest.mark.parametrize("N,H,groups", CASES)
def test_weight_gradient_of_many_rows(dev, N, H, groups):  # noqa: F811
    s, w, dy = normal((N, H), 1, dev), weight(H, F32, dev), normal((N, H), 2, dev)
    rstd = (s.float().square().mean(1) + 1e-6).rsqrt()
    base = torch.randn(H, generator=torch.Generator().manual_seed(3)).to(dev)
    g = moe.rms_norm_backward(dy, s, w, rstd, add=base)
    dw, mag = base.double(), base.double().abs()
    for a in range(0, N, 20000):
        at = slice(a, a + 20000)
        xh = s[at].double() * rstd[at].double()[:, None]
        d = dy[at].double()
        dw, mag = dw + (d * xh).sum(0), mag + (d * xh).abs().sum(0)
        # each row's own gradient, as in test_rms_norm_backward
        e = d * w.double()
        mean, size = (e * xh).mean(1, keepdim=True), (e * xh).abs().mean(1, keepdim=True)
        r = rstd[at].double()[:, None]
        want = r * (e - xh * mean)
        slack = r * (xh.abs() * 64 * U * size + 4 * U * (e.abs() + (xh * mean).abs()))
        assert not ((g.dX[at].double() - want).abs() > slack + 2.0 ** -8 * (want.abs() + slack)).any()
    depth = 64 + 4 * (groups // 64 + 1) + 2 + 3 + 2 + 32 + 1 + 2
    assert not ((g.dweight.double() - dw).abs() > depth * U * mag).any()
    # (what a table row that is overwritten, or a part that is left out, would miss is far beyond that)
    assert float((depth * U * mag).max()) < 0.05 * (N / 3) ** 0.5
    again = moe.rms_norm_backward(dy, s, w, rstd, add=base)
    assert torch.equal(again.dweight, g.dweight) and torch.equal(again.dX, g.dX)


@gpu
@pytest.mark.parametrize("N,H", [(1, 1184), (4101, 1184), (3, 1192), (2500, 1192), (611, 1176)])
@pytest.mark.parametrize("wt", [F32, BF16])
def test_widths_where_the_layout_changes(dev, N, H, wt):  # noqa: F811
    """With three inputs the ring has two places at 1184 columns, and no byte to spare."""
    x, res, w, dy, ds = stream_rows(N, H, 1, dev), stream_rows(N, H, 2, dev), weight(H, wt, dev), normal((N, H), 4, dev), normal((N, H), 5, dev, 0.3)
    n = moe.rms_norm(x, w, residual=res)
    s = n.S.double()
    rstd = (s.square().mean(1) + 1e-6).rsqrt()
    # 40 squares of a lane, 5 steps of a warp, 16 warps at the most: half of that by the root, and the roundings after it
    assert not ((n.rstd.double() - rstd).abs() > 2.0 ** -18 * rstd).any()
    y = s * rstd[:, None] * w.double()
    assert not ((n.Y.double() - y).abs() > (2.0 ** -18 + 2.0 ** -8 * (1 + 2.0 ** -18)) * y.abs()).any()
    g = moe.rms_norm_backward(dy, n.S, w, n.rstd, dS=ds)
    r = n.rstd.double()[:, None]
    xh, d = s * r, dy.double() * w.double()
    mean, size = (d * xh).mean(1, keepdim=True), (d * xh).abs().mean(1, keepdim=True)
    want = r * (d - xh * mean) + ds.double()
    slack = r * (xh.abs() * 64 * U * size + 4 * U * (d.abs() + (xh * mean).abs())) + 2 * U * want.abs()
    assert not ((g.dX.double() - want).abs() > slack + 2.0 ** -8 * (want.abs() + slack)).any()
    dw, mag = (dy.double() * xh).sum(0), (dy.double() * xh).abs().sum(0)
    assert not ((g.dweight.double() - dw).abs() > (64 + 4 + 40 + 2) * U * mag).any()
