"""The selective scan (a decay per channel and state) and its gradients, fp64 --
TEST INFRASTRUCTURE ONLY.  Written from the formulas in numpy, one sequence after
the other and one token after the other.  Shares no code with the library.

Beside the values stand *scales*: c u of the scale (u = 2^-24) bounds the error of
a computation in fp32 whose step sizes, decays, products and sums are each off by a
few u.  With v = dt A a decay a = exp(v) is off by a few u of (1 + |v|) a, since v
is off by a few u of itself; so with S the state of the absolute values, S = a S' +
|b|, the state's scale is H = a H' + (1 + |v|) a S' + |b|: what the state before
was off by, decayed, what its own decay is off by, and its input's roundings.  The
adjoint's G and its absolute value R alike; a product g h has G S + R H.
"""
from __future__ import annotations

import numpy as np

from .block import bounds, dsilu, f64, sigmoid, silu, softplus


def step_sizes(dt, bias=None, limit=None, on=True):
    """Step sizes and their slope by the raw value."""
    raw = f64(dt)
    if not on:
        return raw, np.ones_like(raw)
    v = raw + (0.0 if bias is None else f64(bias))
    lo, hi = (0.0, np.inf) if limit is None else limit
    s = softplus(v)
    return np.clip(s, lo, hi), np.where((s < lo) | (s > hi), 0.0, sigmoid(v))


def _expand(B, C):
    """[T, G, N] -> [T, C, N]."""
    B = f64(B)
    return np.repeat(B, C // B.shape[1], axis=1)


def selective_scan(x, dt, A, B, Cm, lens, D=None, z=None, init=None, **act):
    """x, dt, z [T, C], A [C, N], B, Cm [T, G, N]; returns a dict: y, final, their scales, and every state h [T, C, N]
    with its H and S."""
    x, A = f64(x), f64(A)
    T, C = x.shape
    N = A.shape[1]
    step, _ = step_sizes(dt, **act)
    Be, Ce = _expand(B, C), _expand(Cm, C)
    n = len(lens)
    final = np.zeros((n, C, N)) if init is None else f64(init).copy()
    final_s = np.abs(final)
    h, H, S = (np.zeros((T, C, N)) for _ in range(3))
    for q, (lo, hi) in enumerate(bounds(lens)):
        cur, err, mag = final[q].copy(), np.abs(final[q]), np.abs(final[q])
        for t in range(lo, hi):
            v = step[t][:, None] * A
            a, b = np.exp(v), (step[t] * x[t])[:, None] * Be[t]
            err = a * err + (1 + np.abs(v)) * a * mag + np.abs(b)
            mag = a * mag + np.abs(b)
            cur = a * cur + b
            h[t], H[t], S[t] = cur, err, mag
        final[q], final_s[q] = cur, err
    p = (h * Ce).sum(-1)
    ps = (H * np.abs(Ce)).sum(-1)
    if D is not None:
        p, ps = p + f64(D) * x, ps + np.abs(f64(D) * x)
    gate = 1.0 if z is None else silu(z)
    return dict(y=p * gate, y_s=ps * np.abs(gate), p=p, p_s=ps, final=final, final_s=final_s, h=h, H=H, S=S)


def selective_scan_backward(dy, x, dt, A, B, Cm, lens, D=None, z=None, init=None, dfinal=None, **act):
    """Returns ({name: gradient}, {name: scale})."""
    x, A, dy = f64(x), f64(A), f64(dy)
    T, C = x.shape
    N = A.shape[1]
    G = np.asarray(B).shape[1]
    step, slope = step_sizes(dt, **act)
    Be, Ce = _expand(B, C), _expand(Cm, C)
    f = selective_scan(x, dt, A, B, Cm, lens, D, z, init, **act)
    n = len(lens)
    h0 = np.zeros((n, C, N)) if init is None else f64(init)
    u = dy if z is None else dy * silu(z)
    ua = np.abs(u)
    dinit = np.zeros((n, C, N)) if dfinal is None else f64(dfinal).copy()
    dinit_s = np.abs(dinit)
    dA, dAs = np.zeros((C, N)), np.zeros((C, N))
    s, ss, e, es = (np.zeros((T, C)) for _ in range(4))
    dBe, dBs = np.zeros((T, C, N)), np.zeros((T, C, N))
    for q, (lo, hi) in enumerate(bounds(lens)):
        k, ks, ka = dinit[q].copy(), np.abs(dinit[q]), np.abs(dinit[q])
        for t in range(hi - 1, lo - 1, -1):
            v = step[t][:, None] * A
            a = np.exp(v)
            before = f["h"][t - 1] if t > lo else h0[q]
            Hb = f["H"][t - 1] if t > lo else np.abs(h0[q])
            Sb = f["S"][t - 1] if t > lo else np.abs(h0[q])
            own = ua[t][:, None] * np.abs(Ce[t])
            g, gs, gr = u[t][:, None] * Ce[t] + k, own + ks, own + ka
            s[t], ss[t] = (g * Be[t]).sum(-1), (gs * np.abs(Be[t])).sum(-1)
            dBe[t], dBs[t] = g * (step[t] * x[t])[:, None], gs * np.abs(step[t] * x[t])[:, None]
            k = a * g
            ks, ka = a * gs + (1 + np.abs(v)) * a * gr, a * gr
            w, ws = k * before, ks * Sb + ka * Hb
            e[t], es[t] = (w * A).sum(-1), (ws * np.abs(A)).sum(-1)
            dA += step[t][:, None] * w
            dAs += step[t][:, None] * ws
        dinit[q], dinit_s[q] = k, ks

    def by_group(m):
        return m.reshape(T, G, C // G, N).sum(2)
    skip = 0.0 if D is None else f64(D) * u
    ddt, ddts = (x * s + e) * slope, (np.abs(x) * ss + es) * slope
    grads = dict(dx=step * s + skip, ddt=ddt, dA=dA, dB=by_group(dBe), dC=by_group(f["h"] * u[:, :, None]),
                 dD=(u * x).sum(0), ddt_bias=ddt.sum(0), dinit=dinit)
    scales = dict(dx=step * ss + np.abs(skip), ddt=ddts, dA=dAs, dB=by_group(dBs),
                  dC=by_group(f["H"] * ua[:, :, None]), dD=(ua * np.abs(x)).sum(0), ddt_bias=ddts.sum(0),
                  dinit=dinit_s)
    if z is not None:
        grads["dz"] = dy * f["p"] * dsilu(z)
        # |silu'| <= s (1 + |z|): its two terms without their cancellation
        scales["dz"] = np.abs(dy) * f["p_s"] * sigmoid(z) * (1 + np.abs(f64(z)))
    return grads, scales
