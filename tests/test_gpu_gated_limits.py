"""The gated recurrence at decay factors far over what its gate lets through:
log a = -rate softplus(lam) sigmoid(r) with rate softplus(lam) up to 1e30 and a
gate so nearly closed that the decay is an ordinary one, between rows that forget
everything; against the fp64 oracle, forward, backward and step.

Error counts, in units of 2^-24 of the scale, beside those of the recurrence's
own tests (gate logits up to 6): exp2's argument r log2(e) is off by 1.22 units
of itself (its rounding 1, log2(e)'s 0.22), so sigmoid(r) and log a by 1.22
(|r| - 6) more.  A product of a over a run takes 0.37 of that (|S| exp(-|S|)), the
input weight half, a gradient's factor log a all of it: 3 (|r| - 6) covers them.
A gradient's terms are held divided by the factor k: where they underflow, 2^-150
k is missing a term, the tests' floor of 2^-147 k.
"""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from oracle import block
from block_helpers import offsets, say, up, within
from test_gpu_gated_scan import count, make

pytestmark = pytest.mark.gpu

# rate, lam, r: decays a of about 0.001 to 0.9
CASES = [
    (8.0, (1500.0, 3000.0), (-11.0, -7.5)),
    (3e4, (-0.5, 0.5), (-12.0, -8.5)),
    (1e5, (0.5, 1.5), (-13.0, -10.0)),
    (1e20, (-1.0, 1.0), (-48.0, -44.5)),
    (9e29, (0.0, 0.5), (-71.0, -67.5)),
]


@pytest.mark.parametrize("rate,lam,r", CASES)
def test_large_factors(rate, lam, r):
    say("case: gated large factors", rate, lam, r)
    rate = float(np.float32(rate))
    lens, C = [70, 0, 1, 300, 129], 24
    T = sum(lens)
    d = make(61, lens, C, "f32", decay=lam)
    rng = np.random.default_rng(62)
    d["r"] = rng.uniform(*r, (T, C)).astype(np.float32)
    open_gate = rng.random((T, C)) < 0.1
    d["r"][open_gate] = rng.uniform(-4.0, 4.0, int(open_gate.sum())).astype(np.float32)  # forgets everything
    loga = block.gates(d["x"], d["r"], d["i"], d["lam"], rate)[0]
    ordinary = loga[~open_gate]
    assert (loga[open_gate] < -100).all() and ((ordinary > -12) & (ordinary < -0.01)).mean() > 0.9
    k = rate * float(block.softplus(d["lam"]).max())
    c = count(d, lens, rate) + 3 * (float(np.abs(d["r"]).max()) - 6)
    floor = max(1e-30, 2.0 ** -147 * k)

    args = [up(d[n]) for n in ("x", "r", "i", "lam")]
    kw = dict(rate=rate, init_state=up(d["init"]), cu_seqlens=offsets(lens))
    y, fin, states = ssd.gated_scan(*args, want_states=True, **kw)
    yr, fr, scale = block.gated_scan(d["x"], d["r"], d["i"], d["lam"], lens, rate, d["init"])
    within(y, yr, scale, c, "f32", "y")
    last = np.array([scale[hi - 1] if hi > lo else np.abs(fr[s]) for s, (lo, hi) in enumerate(block.bounds(lens))])
    within(fin, fr, last, c, "f32", "final_state")
    got = ssd.gated_scan_backward(up(d["dy"]), *args, states, dfinal_state=up(d["dfinal"]), **kw)
    ref, sc = block.gated_scan_backward(d["dy"], d["x"], d["r"], d["i"], d["lam"], lens, rate, d["init"], d["dfinal"])
    for name, g in zip(("dx", "dr", "di"), got):
        within(g, ref[name], sc[name], 2 * c + 64, "f32", name, floor)
    within(got[3], ref["dlam"], sc["dlam"], 2 * c + 128 + T / 128, "f32", "dlam", floor * T)
    within(got[4], ref["dinit"], sc["dinit"], c, "f32", "dinit")

    one = {n: d[n][:5] for n in ("x", "r", "i")}
    state = up(d["init"])
    y1 = ssd.gated_scan_step(state, *(up(one[n]) for n in ("x", "r", "i")), args[3], rate=rate)
    yr, fr, s = block.gated_scan(one["x"], one["r"], one["i"], d["lam"], [1] * 5, rate, d["init"])
    within(y1, yr, s, c, "f32", "step")
    within(state, fr, s, c, "f32", "step's state")


def test_factors_over_the_limit_count_as_it():
    say("case: gated factors over the limit")
    L, C, most = 200, 16, float(np.float32(1e30))
    d = make(63, [L], C, "f32")
    d["r"] = np.random.default_rng(64).uniform(-71.0, -67.5, (L, C)).astype(np.float32)
    one = np.full(C, np.log(np.e - 1.0))  # softplus 1
    yr, _, s = block.gated_scan(d["x"], d["r"], d["i"], one, [L], most, d["init"])
    kw = dict(init_state=up(d["init"]))
    c = count({**d, "lam": one}, [L], most) + 3 * (71 - 6)
    for lam, rate in ((1e6, 1e30), (3e38, 8.0), (np.inf, 1.0), (3e38, 3e38)):
        args = [up(d[n]).view(1, L, C) for n in ("x", "r", "i")] + [torch.full((C,), lam, device="cuda")]
        within(ssd.gated_scan(*args, rate=rate, **kw)[0][0], yr, s, c, "f32", "y")
