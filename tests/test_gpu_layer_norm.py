"""The layer norm and its gradients against the fp64 oracle: rows from one wave's
to a workgroup's, with and without the residual, bias and scale, types, a residual
in place, rows far from zero, rows of one value, graphs.

Error counts, in units of 2^-24: a row's sums pass at most 30 additions each, which
moves rstd by 15 + 4 of itself; a handful of products: 64 forward, of what y is a
difference of.  Backward: two means (30 additions) and the same factors: 128; the
sums over rows add one rounding a row.
"""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from oracle import block
from block_helpers import U, down, rounded, say, up, within

pytestmark = pytest.mark.gpu

CASES = [
    # rows, D, dtype, residual's dtype or None, bias, scale
    (1, 8, "f32", "f32", True, True),
    (3, 512, "bf16", "bf16", False, False),
    (5, 520, "bf16", "f32", True, True),
    (1, 776, "f32", None, True, False),
    (33, 1536, "bf16", "bf16", True, True),
    (7, 2048, "bf16", None, True, False),
    (130, 2560, "bf16", "f32", True, True),
    (6, 2816, "f32", "f32", False, True),
    (9, 4096, "bf16", "bf16", True, False),
    (5, 4104, "bf16", None, False, False),
    (4, 5120, "f32", "f32", True, True),
    (3, 8200, "bf16", "f32", True, True),
    (2, 12296, "bf16", "bf16", True, True),
    (2, 16384, "f32", None, True, False),
    (4500, 64, "bf16", "bf16", True, True),
    (777, 136, "f32", None, True, False),
    (600, 264, "bf16", None, True, False),
    (0, 64, "bf16", "bf16", True, True),
    (0, 64, "f32", None, True, False),
    # several rows a workgroup of the gradients, of each kind and width
    (2100, 1536, "bf16", None, True, False),
    (1100, 2560, "f32", None, True, False),
    (2100, 1536, "bf16", "bf16", True, False),
    (2100, 1536, "bf16", "f32", True, True),
    (1100, 5128, "bf16", None, True, False),
    (1100, 5128, "f32", None, False, False),
    (530, 5128, "bf16", "f32", True, False),
    (530, 5128, "bf16", "bf16", True, True),
    (530, 8200, "bf16", None, True, False),
    (530, 8200, "f32", "f32", True, True),
]


@pytest.mark.parametrize("rows,D,dtype,rdtype,biased,scaled", CASES)
def test_layer_norm(rows, D, dtype, rdtype, biased, scaled):
    say("case: layer norm", rows, D, dtype, rdtype, biased, scaled)
    rng = np.random.default_rng(rows + D)
    x = rounded(rng, (rows, D), dtype)
    res = rounded(rng, (rows, D), rdtype, 2.0) if rdtype else None
    w, b = rounded(rng, D, "f32"), rounded(rng, D, "f32") if biased else None
    s = rounded(rng, D, "f32") if scaled else None
    gx, gres, gw, gb, gs = up(x, dtype), up(res, rdtype or "f32"), up(w), up(b), up(s)
    if rdtype:
        y, out, mean, rstd = ssd.add_layer_norm(gx, gres, gw, gb, scale=gs, want_stats=True)
        assert all(torch.equal(p, q) for p, q in zip(ssd.add_layer_norm(gx, gres, gw, gb, scale=gs), (y, out)))
        mag = np.abs(res) + np.abs(x if s is None else s * x)
    else:
        y, mean, rstd = ssd.layer_norm(gx, gw, gb, want_stats=True)
        assert torch.equal(ssd.layer_norm(gx, gw, gb), y)
        out, mag = gx, np.abs(x)
    yr, ur, mr, rr = block.layer_norm(x, w, b, res, s)
    if rdtype:
        within(out, ur, mag, 2, rdtype, "out")
    most = mag.max(-1, keepdims=True, initial=0)
    within(mean, mr, most[:, 0], 64, "f32", "mean")
    # an error of the sum moves rstd by at most its size over the spread
    within(rstd, rr, rr * (1 + most[:, 0] * rr), 64, "f32", "rstd")
    m = np.abs(ur - mr[:, None]) * rr[:, None]
    within(y, yr, ((mag + most) * rr[:, None] * (1 + m) + m) * np.abs(w) + (0 if b is None else np.abs(b)), 64, dtype, "y")

    dy, dout = rounded(rng, (rows, D), dtype), rounded(rng, (rows, D), rdtype or "f32")
    saved = down(out), down(mean), down(rstd)
    if not rdtype:
        got = ssd.layer_norm_backward(up(dy, dtype), gx, gw, mean, rstd, want_dbias=biased)
        ref, sc = block.layer_norm_backward(dy, saved[0], w, *saved[1:])
        for name, g, dt in zip(("dx", "dweight", "dbias"), got, (dtype, "f32", "f32")):
            if g is None:
                assert name == "dbias" and not biased
                continue
            within(g, ref[name], sc[name], 128 + rows, dt, name)
        return
    inplace = gres.clone()
    y2, out2 = ssd.add_layer_norm(gx, inplace, gw, gb, scale=gs, residual_out=inplace)
    assert out2 is inplace and torch.equal(inplace, out) and torch.equal(y2, y)
    for with_out in (True, False):
        kw = dict(x=gx if scaled else None, scale=gs)
        got = ssd.add_layer_norm_backward(up(dy, dtype), out, gw, mean, rstd,
                                          dresidual_out=up(dout, rdtype) if with_out else None, want_dbias=biased, **kw)
        ref, sc = block.layer_norm_backward(dy, saved[0], w, *saved[1:], dout if with_out else None, x, s)
        for name, g, dt in zip(("dx", "dresidual", "dweight", "dbias", "dscale"), got, (dtype, rdtype, "f32", "f32", "f32")):
            if g is None:
                assert name == "dbias" and not biased or name == "dscale" and not scaled
                continue
            within(g, ref[name], sc[name], 128 + rows, dt, name)
    assert (got[0] is got[1]) == (not scaled and dtype == rdtype)
    grad = up(dout, rdtype)
    again = ssd.add_layer_norm_backward(up(dy, dtype), out, gw, mean, rstd, dresidual_out=grad, dresidual=grad, **kw)
    want = ssd.add_layer_norm_backward(up(dy, dtype), out, gw, mean, rstd, dresidual_out=up(dout, rdtype), **kw)
    assert all(p is None or torch.equal(p, q) for p, q in zip(again, want)), "the gradient in place of dresidual_out"


@pytest.mark.parametrize("D", [264, 2560, 8200])
def test_far_from_zero(D):
    """A mean 2^14 times the spread: the distances from it are exact, and y is off by roundings of its own."""
    say("case: layer norm far from zero", D)
    rng = np.random.default_rng(D)
    x = (16384.0 + rng.standard_normal((5, D))).astype(np.float32)
    w, b = rounded(rng, D, "f32"), rounded(rng, D, "f32")
    y, mean, rstd = ssd.layer_norm(up(x), up(w), up(b), want_stats=True)
    yr, _, mr, rr = block.layer_norm(x, w, b)
    within(mean, mr, np.abs(mr), 1, "f32", "mean")
    # the sum of squares loses what the first mean's rounding adds to it, (30 of 2^-24 of 2^14)^2 / 4: nothing
    within(rstd, rr, rr, 64, "f32", "rstd")
    m = np.abs(x - mr[:, None]) * rr[:, None]
    within(y, yr, (1 + m) * np.abs(w) + np.abs(b), 64, "f32", "y")


def test_rows_of_one_value_and_infinities():
    """A row of one value has no spread: y is the bias (eps keeps rstd finite), without eps NaN as the formula's
    0 times infinity; a row that holds NaN or infinity is NaN and does not reach the others."""
    say("case: layer norm not finite")
    D = 264
    x = torch.randn(9, D, device="cuda")
    x[1] = 3.5
    x[2, 5] = float("nan")
    x[4, 7] = float("inf")
    w, b = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    keep = [0, 3, 5, 6, 7, 8]
    clean = ssd.layer_norm(x[keep], w, b)
    y, mean, rstd = ssd.layer_norm(x, w, b, want_stats=True)
    assert torch.equal(y[keep], clean) and torch.equal(y[1], b)
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[4]).any())
    dx, dw, db = ssd.layer_norm_backward(torch.ones_like(x), x, w, mean, rstd)
    assert torch.isfinite(dx[keep + [1]]).all() and torch.isfinite(db).all() and not torch.isfinite(dw).all()
    assert bool(torch.isnan(ssd.layer_norm(x, w, b, eps=0.0)[1]).all())


def test_bf16_rows_round_once():
    """bf16 in, bf16 out: y within half a step of the exact value and the fp32 roundings."""
    say("case: layer norm bf16")
    rng = np.random.default_rng(5)
    x, w = rounded(rng, (64, 1024), "bf16"), np.ones(1024, np.float32)
    y = down(ssd.layer_norm(up(x, "bf16"), up(w)))
    yr = block.layer_norm(x, w)[0]
    assert (np.abs(y - yr) <= 2.0 ** -8 * np.abs(yr) + 64 * U * (8 + np.abs(yr))).all()


def test_in_a_graph():
    say("case: layer norm graph")
    rows, D = 70, 1544
    x, res, dy = (torch.randn(rows, D, device="cuda").bfloat16() for _ in range(3))
    w, b, s = (torch.randn(D, device="cuda") for _ in range(3))

    def all_of(x):
        y, out, mean, rstd = ssd.add_layer_norm(x, res, w, b, scale=s, want_stats=True)
        y2, m2, r2 = ssd.layer_norm(y, w, b, want_stats=True)
        return (y, out, y2, *ssd.layer_norm_backward(dy, y, w, m2, r2),
                *ssd.add_layer_norm_backward(dy, out, w, mean, rstd, dresidual_out=y, x=x, scale=s))
    xin = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_of(xin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_of(xin)
    for k in range(4):
        xin.copy_(x * (k + 1))
        want = all_of(x * (k + 1))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), "replay %d" % k
