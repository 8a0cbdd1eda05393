"""The block operators around the scan, fp64 -- TEST INFRASTRUCTURE ONLY.

The gated linear recurrence, the residual and gated RMS norms and the
gradients of all of them and of the causal conv1d, written from their formulas
in numpy, one sequence after the other and one token after the other.  Shares
no code with the library.

Every function that a tolerance is stated for also returns *scales*: the same
sums with every term replaced by its absolute value, so that a rounding error
of relative size d in the terms is at most d times the scale.
"""
from __future__ import annotations

import numpy as np


def f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def sigmoid(v):
    v = f64(v)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def softplus(v):
    v = f64(v)
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def silu(v):
    return f64(v) * sigmoid(v)


def dsilu(v):
    s = sigmoid(v)
    return s * (1.0 + f64(v) * (1.0 - s))


def bounds(lens):
    c = np.concatenate([[0], np.cumsum(lens)]).astype(int)
    return list(zip(c[:-1], c[1:]))


# ---------------------------------------------------------------- gated recurrence
def gates(x, r, i, lam, rate):
    """log a, a, beta, sigmoid(i) of every token and channel."""
    loga = -rate * softplus(lam) * sigmoid(r)
    return loga, np.exp(loga), np.sqrt(-np.expm1(2.0 * loga)), sigmoid(i)


def gated_scan(x, r, i, lam, lens, rate=8.0, init=None):
    """x, r, i [T, C] with sequence lengths `lens`; returns (y, final, scale)."""
    x, r, i, lam = f64(x), f64(r), f64(i), f64(lam)
    _, a, beta, si = gates(x, r, i, lam, rate)
    b = beta * si * x
    n, C = len(lens), x.shape[1]
    final = np.zeros((n, C)) if init is None else f64(init).copy()
    y, scale = np.zeros_like(x), np.zeros_like(x)
    for q, (lo, hi) in enumerate(bounds(lens)):
        h = final[q].copy()
        s = np.abs(h)
        for t in range(lo, hi):
            h = a[t] * h + b[t]
            s = a[t] * s + np.abs(b[t])
            y[t], scale[t] = h, s
        final[q] = h
    return y, final, scale


def gated_scan_backward(dy, x, r, i, lam, lens, rate=8.0, init=None, dfinal=None):
    """Returns ({name: gradient}, {name: scale})."""
    x, r, i, lam, dy = f64(x), f64(r), f64(i), f64(lam), f64(dy)
    n, C = len(lens), x.shape[1]
    h0 = np.zeros((n, C)) if init is None else f64(init)
    loga, a, beta, si = gates(x, r, i, lam, rate)
    sr = sigmoid(r)
    y, _, habs = gated_scan(x, r, i, lam, lens, rate, init)
    g, gabs = np.zeros_like(x), np.zeros_like(x)
    before, babs = np.zeros_like(x), np.zeros_like(x)
    dinit = np.zeros((n, C)) if dfinal is None else f64(dfinal).copy()
    dinit_s = np.abs(dinit)
    for s, (lo, hi) in enumerate(bounds(lens)):
        q, qa = dinit[s].copy(), np.abs(dinit[s])
        for t in range(hi - 1, lo - 1, -1):
            g[t], gabs[t] = dy[t] + q, np.abs(dy[t]) + qa
            q, qa = a[t] * g[t], a[t] * gabs[t]
            before[t] = y[t - 1] if t > lo else h0[s]
            babs[t] = habs[t - 1] if t > lo else np.abs(h0[s])
        dinit[s], dinit_s[s] = q, qa
    # a^2 / beta diverges as log a goes to 0, where its product with log a goes to 0
    slope = np.divide(a * a * loga, beta, out=np.zeros_like(a), where=beta > 0)
    D = g * (a * before * loga - slope * si * x)
    Ds = gabs * (a * babs * -loga - slope * si * np.abs(x))
    sp = softplus(lam)
    ratio = np.divide(sigmoid(lam), sp, out=np.ones_like(sp), where=sp > 0)
    grads = dict(dx=g * beta * si, dr=D * (1.0 - sr), di=g * beta * x * si * (1.0 - si), dlam=D.sum(0) * ratio,
                 dinit=dinit)
    scales = dict(dx=gabs * beta * si, dr=Ds, di=gabs * beta * np.abs(x) * si, dlam=Ds.sum(0) * ratio, dinit=dinit_s)
    return grads, scales


# ---------------------------------------------------------------- norms
def add_rms_norm(x, residual, weight, scale=None, eps=1e-5):
    x, u = f64(x), f64(residual)
    u = u + (x if scale is None else f64(scale) * x)
    rstd = 1.0 / np.sqrt(np.mean(u * u, axis=-1) + eps)
    return u * rstd[..., None] * f64(weight), u, rstd


def add_rms_norm_backward(dy, out, weight, rstd, dout=None, x=None, scale=None):
    dy, w, rstd = f64(dy), f64(weight), f64(rstd)[..., None]
    m = f64(out) * rstd
    wd = dy * w
    c, cs = (np.mean(v, axis=-1, keepdims=True) for v in (wd * m, np.abs(wd * m)))
    extra = np.zeros_like(m) if dout is None else f64(dout)
    dres = extra + rstd * (wd - m * c)
    dres_s = np.abs(extra) + rstd * (np.abs(wd) + np.abs(m) * cs)
    s = 1.0 if scale is None else f64(scale)
    axes = tuple(range(m.ndim - 1))
    grads = dict(dx=dres * s, dresidual=dres, dweight=(dy * m).sum(axes))
    scales = dict(dx=dres_s * np.abs(s), dresidual=dres_s, dweight=np.abs(dy * m).sum(axes))
    if scale is not None:
        grads["dscale"] = (dres * f64(x)).sum(axes)
        scales["dscale"] = (dres_s * np.abs(f64(x))).sum(axes)
    return grads, scales


def gated_rms_norm(x, z, weight, groups=1, eps=1e-5, norm_first=False):
    x, z, w = f64(x), f64(z), f64(weight)
    v = x if norm_first else x * silu(z)
    vg = v.reshape(v.shape[:-1] + (groups, v.shape[-1] // groups))
    rstd = 1.0 / np.sqrt(np.mean(vg * vg, axis=-1) + eps)
    y = (vg * rstd[..., None]).reshape(v.shape) * w
    return (y * silu(z) if norm_first else y), rstd


def gated_rms_norm_backward(dy, x, z, weight, groups=1, eps=1e-5, norm_first=False):
    dy, x, z, w = f64(dy), f64(x), f64(z), f64(weight)
    _, rstd = gated_rms_norm(x, z, w, groups, eps, norm_first)
    gate = silu(z)

    def grouped(v):
        return v.reshape(v.shape[:-1] + (groups, v.shape[-1] // groups))
    v = x if norm_first else x * gate
    m = grouped(v) * rstd[..., None]
    d = dy * gate if norm_first else dy
    wd = grouped(d * w)
    c, cs = (np.mean(t, axis=-1, keepdims=True) for t in (wd * m, np.abs(wd * m)))
    dv = (rstd[..., None] * (wd - m * c)).reshape(v.shape)
    dvs = (rstd[..., None] * (np.abs(wd) + np.abs(m) * cs)).reshape(v.shape)
    m = m.reshape(v.shape)
    axes = tuple(range(m.ndim - 1))
    # |silu'| <= s (1 + |z|): its two terms without their cancellation
    slope = sigmoid(z) * (1.0 + np.abs(z))
    if norm_first:
        dx, dxs, dz, dzs = dv, dvs, dy * m * w * dsilu(z), np.abs(dy * m * w) * slope
    else:
        dx, dxs, dz, dzs = dv * gate, dvs * np.abs(gate), dv * x * dsilu(z), dvs * np.abs(x) * slope
    return (dict(dx=dx, dz=dz, dweight=(d * m).sum(axes)), dict(dx=dxs, dz=dzs, dweight=np.abs(d * m).sum(axes)))


# ---------------------------------------------------------------- conv1d gradients
def causal_conv1d_backward(dy, x, weight, bias, lens, state=None, dfinal=None, activation=True):
    """dy, x [T, C], weight [C, K], state and dfinal [n, K-1, C] or None."""
    dy, x, w = f64(dy), f64(x), f64(weight)
    C, K = w.shape
    n = len(lens)
    b = np.zeros(C) if bias is None else f64(bias)
    dx, dxs = np.zeros_like(x), np.zeros_like(x)
    dw, dws, db, dbs = np.zeros((C, K)), np.zeros((C, K)), np.zeros(C), np.zeros(C)
    dst, dsts = np.zeros((n, K - 1, C)), np.zeros((n, K - 1, C))
    for s, (lo, hi) in enumerate(bounds(lens)):
        L = hi - lo
        st = np.zeros((K - 1, C)) if state is None else f64(state)[s]
        xp = np.concatenate([st, x[lo:hi]])
        v, va = b + np.zeros((L, C)), np.abs(b) + np.zeros((L, C))
        for k in range(K):
            v = v + w[:, k] * xp[k:k + L]
            va = va + np.abs(w[:, k] * xp[k:k + L])
        dv = dy[lo:hi] * (dsilu(v) if activation else 1.0)
        # an error in v of relative size d of va moves silu' by at most d va / 2; its own terms are below 1 + |v|
        dva = np.abs(dy[lo:hi]) * (sigmoid(v) * (1.0 + np.abs(v)) + 0.5 * va if activation else 1.0)
        gp, gps = np.zeros_like(xp), np.zeros_like(xp)
        for k in range(K):
            gp[k:k + L] += w[:, k] * dv
            gps[k:k + L] += np.abs(w[:, k]) * dva
            dw[:, k] += (dv * xp[k:k + L]).sum(0)
            dws[:, k] += (dva * np.abs(xp[k:k + L])).sum(0)
        if dfinal is not None:
            gp[L:] += f64(dfinal)[s]
            gps[L:] += np.abs(f64(dfinal)[s])
        db += dv.sum(0)
        dbs += dva.sum(0)
        dst[s], dsts[s] = gp[:K - 1], gps[:K - 1]
        dx[lo:hi], dxs[lo:hi] = gp[K - 1:], gps[K - 1:]
    return (dict(dx=dx, dweight=dw, dbias=db, dstate=dst), dict(dx=dxs, dweight=dws, dbias=dbs, dstate=dsts))
