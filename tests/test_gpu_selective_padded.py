"""Infinities where the states do not fill a wave's quarters (a lane then holds states
that are not there): y, the states and the gradients are the formula's, infinities and
all, as where they do.  Every factor is positive and no decay underflows, so that the
formula says which values are infinite."""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import offsets, say, up

pytestmark = pytest.mark.gpu
INF = float("inf")
NS = [1, 2, 3, 5, 7, 11, 13, 16, 20, 31, 37, 64]


def a_case(N, dtype, lens, C=24, G=1):
    rng = np.random.default_rng(N)
    T = sum(lens)
    u = {k: rng.uniform(0.25, 1.0, s).astype(np.float32) for k, s in dict(
        x=(T, C), B=(T, G, N), Cm=(T, G, N), z=(T, C), dy=(T, C)).items()}
    d = {k: up(v, dtype) for k, v in u.items()}
    d["dt"] = up(rng.uniform(0.01, 0.1, (T, C)).astype(np.float32), dtype)
    d["A"] = up(-rng.uniform(0.1, 1.0, (C, N)).astype(np.float32))
    d["D"] = up(rng.uniform(0.25, 1.0, C).astype(np.float32))
    d["cu"] = offsets(lens)
    return d


def scan(d, **kw):
    return ssd.selective_scan(d["x"], d["dt"], d["A"], d["B"], d["Cm"], D=d["D"], z=d["z"], cu_seqlens=d["cu"], **kw)


def back(d, states, **kw):
    return ssd.selective_scan_backward(d["dy"], d["x"], d["dt"], d["A"], d["B"], d["Cm"], states, D=d["D"], z=d["z"],
                                       cu_seqlens=d["cu"], **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", NS)
def test_forward(N, dtype):
    say("case: selective scan, padded states", N, dtype)
    lens = [61, 150, 3]
    d = a_case(N, dtype, lens)
    y0, f0, _ = scan(d, want_states=True)
    for name, at in (("x", 70), ("x", 60), ("dt", 75), ("dt", 213)):
        bad = dict(d)
        bad[name] = d[name].clone()
        bad[name][at, 5] = INF
        y, f, states = scan(bad, want_states=True)
        s = 0 if at < 61 else 1 if at < 211 else 2
        end = sum(lens[:s + 1])
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[at:end, 5] = True
        assert torch.equal(y[~hit], y0[~hit]), (name, at)
        assert (y[hit] == INF).all(), (name, at, y[hit])
        keep = torch.ones_like(f, dtype=torch.bool)
        keep[s, 5] = False
        assert torch.equal(f[keep], f0[keep]) and (f[~keep] == INF).all(), (name, at)
        # the tokens that came before, from the states that were saved
        got, want = back(bad, states), back(d, scan(d, want_states=True)[2])
        for k in (0, 1, 6):  # dx, ddt, dz: of the other channels
            other = [c for c in range(24) if c != 5]
            assert torch.equal(got[k][:, other], want[k][:, other]), (name, at, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", NS)
def test_gradients(N, dtype):
    """An infinite dy, or an infinite input of the gate: its own token's and every earlier token's dx is infinite, and
    every earlier input's; the sums over states are not NaN by states that are not there."""
    say("case: selective scan, padded states, gradients", N, dtype)
    lens = [61, 150, 3]
    d = a_case(N, dtype, lens)
    states = scan(d, want_states=True)[2]
    want = back(d, states)
    other = [c for c in range(24) if c != 5]
    for name, at in (("dy", 190), ("dy", 61), ("dy", 213), ("z", 100)):
        bad = dict(d)
        bad[name] = d[name].clone()
        bad[name][at, 5] = INF
        got = back(bad, states)
        s = 0 if at < 61 else 1 if at < 211 else 2
        first = sum(lens[:s])
        dx, dz, dinit = got[0], got[6], got[8]
        hit = torch.zeros_like(dx, dtype=torch.bool)
        hit[first:at + 1, 5] = True
        assert (dx[hit] == INF).all(), (name, at, dx[hit])
        assert torch.equal(dx[~hit], want[0][~hit]), (name, at)
        assert (dinit[s, 5] == INF).all() and torch.equal(dinit[:, other], want[8][:, other]), (name, at)
        for k in (1, 6):
            assert torch.equal(got[k][:, other], want[k][:, other]), (name, at, k)
        if name == "dy":
            assert dz[at, 5] == INF
            rest = torch.arange(dz.shape[0], device="cuda") != at
            assert torch.equal(dz[rest], want[6][rest])
        # dB of the infinite adjoint, for every state
        assert (got[3][first:at + 1] == INF).all() and (got[4][at] == INF).all(), (name, at)
        out = [t for t in range(sum(lens)) if t < first or t > at]
        assert torch.equal(got[3][out], want[3][out]) and torch.equal(got[4][out], want[4][out])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinite_inputs_behind(dtype):
    """An infinite x: the gradients of its sequence that the infinite states do not reach stay as they were, and dz,
    which reads the states, is the infinity itself."""
    say("case: selective scan, padded states, infinite x", dtype)
    lens = [61, 150, 3]
    for N in NS:
        d = a_case(N, dtype, lens)
        want = back(d, scan(d, want_states=True)[2])
        bad = dict(d)
        bad["x"] = d["x"].clone()
        bad["x"][130, 5] = INF
        got = back(bad, scan(bad, want_states=True)[2])
        assert (got[6][130:211, 5] == INF).all(), N
        assert torch.equal(got[6][:130], want[6][:130]), N
        assert torch.equal(got[0], want[0]), N  # dx does not read x or the states
        assert (got[4][130:211] == INF).all() and torch.equal(got[4][:130], want[4][:130]), N
