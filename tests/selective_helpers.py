"""Inputs and comparisons of the selective scan's GPU tests.

An fp32 result may be off by c units u = 2^-24 of its scale (oracle/selective.py),
c counting what the scale leaves open:
  the step size: 4 u of softplus, 1 of its argument's rounding, which moves it by at
  most |argument| <= 8 of its u: 13;  an exponent dt A log2(e): 13 + 3;  a decay: 16
  of (1 + |v|) u and 1 of the exponential;  dt x B: 15;  the addition: 1   -> 32
  a sum over 64 states: 16 + 2 additions;  silu 17 + 6 (block_helpers)   -> 32 + 48
  a gradient adds the gate's silu' (23), the adjoint's own additions and products
  and the slope (6)                                                     -> 128
  a sum over rows adds one rounding a row of an item, one over channels 4 + 8 and
  one a block of 128 channels.
A bf16 output adds half a step, 2^-8 of the value.
"""
from __future__ import annotations

import numpy as np
import torch

from block_helpers import DTYPES, in_wider, offsets, rounded, up, within

STATE, OUT, GRAD = 32, 80, 128


def make(rng, lens, C, N, G, dtype, gated=True, skip=True, act="bias", init=True, a_scale=1.0):
    """Host values of a case, as the dtype holds them."""
    T, n = int(np.sum(lens)), len(lens)
    v = dict(x=rounded(rng, (T, C), dtype), B=rounded(rng, (T, G, N), dtype), Cm=rounded(rng, (T, G, N), dtype),
             A=(-np.exp(rng.uniform(-2.0, 2.5, (C, N))) * a_scale).astype(np.float32),
             z=rounded(rng, (T, C), dtype) if gated else None,
             D=rounded(rng, C, "f32") if skip else None,
             init=rounded(rng, (n, C, N), "f32") if init else None)
    kw = {}
    if act == "none":
        v["dt"] = torch.from_numpy(rng.uniform(0.01, 0.3, (T, C)).astype(np.float32)).to(DTYPES[dtype]).float().numpy()
        kw["on"] = False
    else:
        v["dt"] = rounded(rng, (T, C), dtype, 1.0, 3.0)
        if act != "plain":
            kw["bias"] = rounded(rng, C, "f32", 1.0, 3.0) - 1.0
        if act == "clamp":
            kw["limit"] = (0.1, 0.5)
    return v, kw


def options(kw):
    """The binding's keywords for an activation."""
    if not kw.get("on", True):
        return {}
    return dict(dt_softplus=True, dt_bias=up(kw.get("bias")), dt_limit=kw.get("limit"))


class Case:
    """Device tensors of a case, dense [n, L, ...] where the lengths are equal and `dense` says so."""

    def __init__(self, v, kw, lens, dtype, dense, wide=False):
        self.lead = (len(lens), lens[0]) if dense else (int(np.sum(lens)),)
        self.dtype, self.dense, self.lens = dtype, dense, lens
        self.kw = options(kw)

        def rows(a, spare=0):
            if a is None:
                return None
            a = a.reshape(self.lead + a.shape[1:])
            if not wide:
                return up(a, dtype)
            if spare:  # B and C: two states' width in front, an odd rest behind
                flat = in_wider(a.reshape(self.lead + (a.shape[-2] * a.shape[-1],)), dtype, self.lead, spare, spare + 1)
                return flat.unflatten(-1, a.shape[-2:])
            return in_wider(a, dtype, self.lead)
        self.x, self.dt, self.z = rows(v["x"]), rows(v["dt"]), rows(v["z"])
        self.B, self.C = rows(v["B"], 2), rows(v["Cm"], 3)
        self.A, self.D, self.init = up(v["A"]), up(v["D"]), up(v["init"])
        self.cu = None if dense else offsets(lens)
        self.args = (self.x, self.dt, self.A, self.B, self.C)
        self.kw.update(D=self.D, z=self.z, init_state=self.init, cu_seqlens=self.cu)

    def rows(self, a, dtype=None):
        """Host rows [T, ...] as the case's device tensor."""
        return up(a.reshape(self.lead + a.shape[1:]), dtype or self.dtype)


def flat(t, like):
    return t.reshape(like.shape)


__all__ = ["STATE", "OUT", "GRAD", "make", "options", "Case", "flat", "within", "up", "rounded", "DTYPES"]
