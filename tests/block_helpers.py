"""Helpers of the block operators' GPU tests.

An fp32 result may be off by c units u = 2^-24 of its *scale* (the same sums
with every term's absolute value, from the oracle), c counting the roundings
and the hardware functions' errors on the way; a bf16 output adds half a step,
2^-8 of the value.  The counts behind each c stand at the tests.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def say(*a):
    print(*a, flush=True)


def rounded(rng, shape, dtype, scale=1.0, clip=6.0):
    """Values that `dtype` holds, as fp32 on the host."""
    a = np.clip(rng.standard_normal(shape) * scale, -clip, clip).astype(np.float32)
    return torch.from_numpy(a).to(DTYPES[dtype]).float().numpy()


def up(a, dtype="f32"):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DTYPES[dtype]).cuda()


def down(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, scale, c, dtype, what, floor=1e-30):
    """|got - ref| <= c u scale + (bf16) 2^-8 |ref|, everywhere.  Below `floor` nothing is asked; 1e-30: the kernels'
    smallest decay is 1e-37 where the formula's underflows, and a gradient multiplies it by up to 1e4 (the largest
    -log a) and by a state and an adjoint, each below 1e1 here."""
    g, r = down(got), np.asarray(ref, np.float64)
    assert g.shape == r.shape, (what, g.shape, r.shape)
    if not g.size:
        return
    tol = c * U * np.broadcast_to(scale, r.shape)
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(r) + tol)
    off = np.abs(g - r)
    bad = ~(off <= tol + floor)
    assert not bad.any(), "%s: %d of %d off, first at %s: %r for %r (tolerance %.3g)" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0], r[bad][0], tol[bad][0])


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def in_wider(a, dtype, lead, before=8, after=16):
    """The values of a as a column range of a wider tensor (filled with NaN elsewhere)."""
    w = torch.full(tuple(lead) + (before + a.shape[-1] + after,), float("nan"), dtype=DTYPES[dtype], device="cuda")
    v = w[..., before:before + a.shape[-1]]
    v.copy_(up(a, dtype).view(v.shape))
    return v
