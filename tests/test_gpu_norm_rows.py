"""The norms' gradients where a team of lanes takes several rows one after the
other (more rows than the backward pass's workgroups hold at once): every width
of a team, both types, groups, both orders of gate and norm, and the gradient in
place of the one it is added to.

Error counts, in units of 2^-24 of the scale: 128 a row, as in the norms' own
tests; a sum over rows passes the rows of a team, 6 steps to the workgroup's sum,
then parts / 64 + 16 of the partial sums.
"""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from mamba_ssd_chunked_02_amd import block_ops as ops
from oracle import block
from block_helpers import rounded, say, up, within

pytestmark = pytest.mark.gpu


def rows_of_a_team(rows, D, groups):
    """Workgroups along the rows (their partial sums are the workspace), and the rows that a team takes."""
    torch.cuda.init()
    ops._lib()
    parts = ops._norm_bytes(rows, D, groups) // (8 * D)
    n = D // groups
    teams = parts * (1 if n > 512 else 256 // (8 if n <= 64 else 16 if n <= 128 else 32 if n <= 256 else 64))
    assert rows > 2 * teams, "%d rows in %d teams: none takes three" % (rows, teams)
    return parts, -(-rows // teams)


RESIDUAL = [
    # rows, D, dtype, residual's dtype, scaled
    (70001, 64, "bf16", "bf16", True),
    (36003, 128, "f32", "f32", True),
    (18005, 248, "bf16", "f32", False),
    (9001, 512, "bf16", "bf16", False),
    (3001, 1536, "bf16", "f32", True),
    (3001, 1544, "bf16", "bf16", True),
    (1101, 4096, "f32", "f32", True),
    (601, 8192, "bf16", "bf16", True),
    (603, 8184, "bf16", "f32", True),
    (530, 16384, "bf16", "bf16", True),
    (530, 16384, "f32", "f32", False),
]


@pytest.mark.parametrize("rows,D,dtype,rdtype,scaled", RESIDUAL)
def test_residual_norm(rows, D, dtype, rdtype, scaled):
    say("case: residual norm of many rows", rows, D, dtype, rdtype, scaled)
    parts, each = rows_of_a_team(rows, D, 1)
    rng = np.random.default_rng(rows + D)
    x, res = rounded(rng, (rows, D), dtype), rounded(rng, (rows, D), rdtype, 2.0)
    w, s = rounded(rng, D, "f32"), rounded(rng, D, "f32") if scaled else None
    gx, gw, gs = up(x, dtype), up(w), up(s)
    _, out, rstd = ssd.add_rms_norm(gx, up(res, rdtype), gw, scale=gs, want_rstd=True)
    dy, dout = rounded(rng, (rows, D), dtype), rounded(rng, (rows, D), rdtype)
    kw = dict(x=gx if scaled else None, scale=gs)
    got = ssd.add_rms_norm_backward(up(dy, dtype), out, gw, rstd, dresidual_out=up(dout, rdtype), **kw)
    saved, savedr = out.double().cpu().numpy(), rstd.double().cpu().numpy()
    ref, sc = block.add_rms_norm_backward(dy, saved, w, savedr, dout, x, s)
    sums = 128 + each + 6 + parts / 64 + 16
    for name, g, dt, c in zip(("dx", "dresidual", "dweight", "dscale"), got, (dtype, rdtype, "f32", "f32"),
                              (128, 128, sums, sums)):
        if name != "dscale" or scaled:
            within(g, ref[name], sc[name], c, dt, name)
    if dtype != rdtype:
        return
    # dx in place of dresidual_out, which is dy as well
    g1, g2 = up(dy, dtype), up(dy, dtype)
    want = ssd.add_rms_norm_backward(g1, out, gw, rstd, dresidual_out=g1, **kw)
    again = ssd.add_rms_norm_backward(g2, out, gw, rstd, dresidual_out=g2, dx=g2, **kw)
    assert again[0] is g2 and all(a is None or torch.equal(a, b) for a, b in zip(again, want))


GATED = [
    # rows, D, groups, dtype, x's dtype, norm first
    (70001, 64, 1, "bf16", "bf16", False),
    (9001, 512, 8, "bf16", "f32", True),
    (9003, 512, 4, "f32", "f32", False),
    (18005, 248, 1, "bf16", "bf16", True),
    (9001, 1024, 2, "bf16", "bf16", False),
    (701, 8192, 8, "bf16", "bf16", False),
    (3001, 1536, 1, "bf16", "f32", False),
    (1101, 4096, 1, "f32", "f32", True),
    (601, 8192, 1, "bf16", "bf16", True),
    (530, 16384, 1, "bf16", "bf16", False),
    (530, 12296, 1, "f32", "f32", True),
]


@pytest.mark.parametrize("rows,D,groups,dtype,xdtype,first", GATED)
def test_gated_norm(rows, D, groups, dtype, xdtype, first):
    say("case: gated norm of many rows", rows, D, groups, dtype, xdtype, first)
    parts, each = rows_of_a_team(rows, D, groups)
    rng = np.random.default_rng(rows + D)
    x, z, w = rounded(rng, (rows, D), xdtype), rounded(rng, (rows, D), dtype, 2.0), rounded(rng, D, "f32")
    dy = rounded(rng, (rows, D), dtype)
    kw = dict(groups=groups, norm_before_gate=first)
    gx, gz, gw = up(x, xdtype), up(z, dtype), up(w)
    _, rstd = ssd.gated_rms_norm(gx, gz, gw, want_rstd=True, **kw)
    got = ssd.gated_rms_norm_backward(up(dy, dtype), gx, gz, gw, rstd, **kw)
    ref, sc = block.gated_rms_norm_backward(dy, x, z, w, groups, norm_first=first)
    for name, g, dt, c in zip(("dx", "dz", "dweight"), got, (xdtype, dtype, "f32"),
                              (128, 128, 128 + each + 6 + parts / 64 + 16)):
        within(g, ref[name], sc[name], c, dt, name)
