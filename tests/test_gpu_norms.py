"""The residual and gated RMS norms and their gradients against the fp64
oracle: rows from one wave's to a workgroup's, groups, both orders of gate and
norm, types, in-place residuals, column ranges, rows of zeros, graphs.

Error counts, in units of 2^-24 of the scale: a row's sum of squares passes at
most 30 additions, so rstd is off by 15 + 4; silu by 17 + 6; a handful of
products: 64 forward.  Backward: the row's mean (30 additions) and the same
factors: 128; the sums over rows add one rounding a row.
"""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from oracle import block
from block_helpers import DTYPES, in_wider, rounded, say, up, within

pytestmark = pytest.mark.gpu

RESIDUAL = [
    # rows, D, dtype, residual's dtype, scaled
    (1, 8, "f32", "f32", True),
    (3, 512, "bf16", "bf16", False),
    (5, 520, "bf16", "f32", True),
    (1, 776, "f32", "f32", False),
    (33, 1536, "bf16", "bf16", True),
    (7, 2048, "bf16", "f32", False),
    (130, 2560, "bf16", "f32", True),
    (6, 2816, "f32", "f32", True),
    (9, 4096, "bf16", "bf16", True),
    (5, 4104, "bf16", "bf16", False),
    (4, 5120, "f32", "f32", True),
    (3, 8200, "bf16", "f32", True),
    (2, 12296, "bf16", "bf16", True),
    (2, 16384, "f32", "f32", True),
    (4500, 64, "bf16", "bf16", True),
    (0, 64, "bf16", "bf16", True),
]


@pytest.mark.parametrize("rows,D,dtype,rdtype,scaled", RESIDUAL)
def test_residual_norm(rows, D, dtype, rdtype, scaled):
    say("case: residual norm", rows, D, dtype, rdtype, scaled)
    rng = np.random.default_rng(rows + D)
    x, res = rounded(rng, (rows, D), dtype), rounded(rng, (rows, D), rdtype, 2.0)
    w = rounded(rng, D, "f32")
    s = rounded(rng, D, "f32") if scaled else None
    gx, gres, gw, gs = up(x, dtype), up(res, rdtype), up(w), up(s)
    y, out, rstd = ssd.add_rms_norm(gx, gres, gw, scale=gs, want_rstd=True)
    yr, ur, rr = block.add_rms_norm(x, res, w, s)
    mag = np.abs(res) + np.abs(x if s is None else s * x)
    within(out, ur, mag, 2, rdtype, "out")
    within(rstd, rr, rr, 64, "f32", "rstd")
    # an error of the sum moves y directly and through rstd
    within(y, yr, (mag + mag.max(-1, keepdims=True, initial=0)) * rr[:, None] * np.abs(w), 64, dtype, "y")
    inplace = gres.clone()
    y2, out2 = ssd.add_rms_norm(gx, inplace, gw, scale=gs, residual_out=inplace)
    assert out2 is inplace and torch.equal(inplace, out) and torch.equal(y2, y)

    dy, dout = rounded(rng, (rows, D), dtype), rounded(rng, (rows, D), rdtype)
    saved, savedr = out.double().cpu().numpy(), rstd.double().cpu().numpy()
    for with_out in (True, False):
        got = ssd.add_rms_norm_backward(up(dy, dtype), out, gw, rstd, dresidual_out=up(dout, rdtype) if with_out else None,
                                        x=gx if scaled else None, scale=gs)
        ref, sc = block.add_rms_norm_backward(dy, saved, w, savedr, dout if with_out else None, x, s)
        for name, g, dt in zip(("dx", "dresidual", "dweight", "dscale"), got, (dtype, rdtype, "f32", "f32")):
            if name == "dscale" and not scaled:
                assert g is None
                continue
            within(g, ref[name], sc[name], 128 + rows, dt, name)
    assert (got[0] is got[1]) == (not scaled and dtype == rdtype)
    grad = up(dout, rdtype)
    again = ssd.add_rms_norm_backward(up(dy, dtype), out, gw, rstd, dresidual_out=grad, dresidual=grad,
                                      x=gx if scaled else None, scale=gs)
    want = ssd.add_rms_norm_backward(up(dy, dtype), out, gw, rstd, dresidual_out=up(dout, rdtype),
                                     x=gx if scaled else None, scale=gs)
    assert all(a is None or torch.equal(a, b) for a, b in zip(again, want)), "the gradient in place of dresidual_out"


GATED = [
    # rows, D, groups, dtype, x's dtype, norm first, wide
    (1, 8, 1, "f32", "f32", False, False),
    (3, 64, 8, "bf16", "f32", False, True),
    (5, 520, 1, "bf16", "bf16", True, False),
    (33, 1536, 1, "bf16", "f32", False, False),
    (6, 1536, 4, "f32", "f32", True, True),
    (11, 8192, 8, "bf16", "bf16", False, True),
    (4, 5120, 1, "bf16", "f32", False, False),
    (3, 5120, 1, "bf16", "bf16", True, False),
    (3, 8192, 1, "f32", "f32", False, False),
    (2, 16384, 1, "bf16", "bf16", True, False),
    (2, 24576, 2, "bf16", "bf16", False, False),
    (3000, 40, 5, "bf16", "bf16", False, False),
    (0, 64, 2, "bf16", "f32", False, False),
]


@pytest.mark.parametrize("rows,D,groups,dtype,xdtype,first,wide", GATED)
def test_gated_norm(rows, D, groups, dtype, xdtype, first, wide):
    say("case: gated norm", rows, D, groups, dtype, xdtype, first, wide)
    rng = np.random.default_rng(rows + D)
    x, z, w = rounded(rng, (rows, D), xdtype), rounded(rng, (rows, D), dtype, 2.0), rounded(rng, D, "f32")
    gx = in_wider(x, xdtype, (rows,)) if wide else up(x, xdtype)
    gz = in_wider(z, dtype, (rows,), 16, 0) if wide else up(z, dtype)
    kw = dict(groups=groups, norm_before_gate=first)
    y, rstd = ssd.gated_rms_norm(gx, gz, up(w), want_rstd=True, **kw)
    yr, rr = block.gated_rms_norm(x, z, w, groups, norm_first=first)
    within(rstd, rr, rr, 64, "f32", "rstd")
    within(y, yr, np.abs(yr), 64 + 23, dtype, "y")
    assert torch.equal(ssd.gated_rms_norm(gx, gz, up(w), **kw), y)
    dy = rounded(rng, (rows, D), dtype)
    given = {}
    if wide:
        given = {"dx": torch.empty((rows, D + 24), dtype=DTYPES[xdtype], device="cuda")[:, 8:D + 8],
                 "dz": torch.empty((rows, 2 * D), dtype=DTYPES[dtype], device="cuda")[:, D:]}
    got = ssd.gated_rms_norm_backward(up(dy, dtype), gx, gz, up(w), rstd, **kw, **given)
    ref, sc = block.gated_rms_norm_backward(dy, x, z, w, groups, norm_first=first)
    for name, g, dt in zip(("dx", "dz", "dweight"), got, (xdtype, dtype, "f32")):
        within(g, ref[name], sc[name], 128 + rows, dt, name)


def test_rows_of_zeros_and_infinities():
    """A row of zeros is finite (eps keeps rstd so); without eps it is NaN, as the formula's 0 / 0; a row
    that holds NaN or infinity does not reach the others; a gate that closes far below 0 gives 0."""
    say("case: norms not finite")
    D = 264
    x, z = torch.randn(9, D, device="cuda"), torch.randn(9, D, device="cuda")
    x[1] = 0
    x[2, 5] = float("nan")
    x[4, 7] = float("inf")
    z[5] = -1e4
    w = torch.ones(D, device="cuda")
    clean = ssd.gated_rms_norm(x[[0, 3, 6, 7, 8]], z[[0, 3, 6, 7, 8]], w)
    y, rstd = ssd.gated_rms_norm(x, z, w, want_rstd=True)
    assert torch.equal(y[[0, 3, 6, 7, 8]], clean)
    assert not y[1].any() and not y[5].any() and bool(torch.isnan(y[2]).all())
    dx, dz, _ = ssd.gated_rms_norm_backward(torch.ones_like(x), x, z, w, rstd)
    keep = [0, 1, 3, 5, 6, 7, 8]
    assert torch.isfinite(dx[keep]).all() and torch.isfinite(dz[keep]).all()
    y, out = ssd.add_rms_norm(x, torch.zeros_like(x), w, eps=0.0)
    assert bool(torch.isnan(y[1]).all()) and torch.isfinite(y[0]).all()


def test_norms_in_a_graph():
    say("case: norms graph")
    rows, D = 70, 1544
    x, res, z, dy = (torch.randn(rows, D, device="cuda").bfloat16() for _ in range(4))
    w, s = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")

    def all_of(x):
        y, out, rstd = ssd.add_rms_norm(x, res, w, scale=s, want_rstd=True)
        g, r2 = ssd.gated_rms_norm(x, z, w, want_rstd=True)
        return (y, out, g, *ssd.add_rms_norm_backward(dy, out, w, rstd, dresidual_out=y, x=x, scale=s),
                *ssd.gated_rms_norm_backward(dy, x, z, w, r2))
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
        assert all(torch.equal(a, b) for a, b in zip(out, want)), "replay %d" % k
