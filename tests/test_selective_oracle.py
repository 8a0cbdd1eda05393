"""The fp64 oracle of the selective scan against itself: its gradients against
central differences of its forward pass, its recurrence against the closed form at
constant inputs, and against the SSD scan's oracle where all states decay alike."""
import numpy as np
import pytest

import oracle
from oracle import block, selective
from test_block_oracle import differences

RNG = np.random.default_rng


def test_closed_form():
    """One state, constant inputs: h_t = a^t h_0 + dt x B (1 - a^t) / (1 - a)."""
    L, C = 40, 3
    A = -np.array([[0.1], [1.0], [3.0]])
    one = np.ones((L, C))
    f = selective.selective_scan(2 * one, 0.25 * one, A, np.full((L, 1, 1), 3.0), np.full((L, 1, 1), -1.0), [L],
                                 init=np.full((1, C, 1), 5.0), on=False)
    a, t = np.exp(0.25 * A[:, 0]), np.arange(1, L + 1)[:, None]
    h = a ** t * 5 + 0.25 * 2 * 3 * (1 - a ** t) / (1 - a)
    np.testing.assert_allclose(f["y"], -h, rtol=1e-12)
    np.testing.assert_allclose(f["final"][0, :, 0], h[-1], rtol=1e-12)


def test_equal_decays_are_the_ssd_scan():
    rng, L, H, P, N = RNG(3), 30, 2, 4, 5
    x, B, C = rng.standard_normal((1, L, H, P)), rng.standard_normal((1, L, 1, N)), rng.standard_normal((1, L, 1, N))
    dt, A, D = rng.uniform(0.01, 0.5, (1, L, H)), -rng.uniform(0.1, 2, H), rng.standard_normal(H)
    h0 = rng.standard_normal((1, H, P, N))
    x, dt, A, B, C, D, h0 = (v.astype(np.float32) for v in (x, dt, A, B, C, D, h0))
    y, fin = oracle.scan(x, dt, A, B, C, D, init=h0)
    f = selective.selective_scan(x[0].reshape(L, -1), np.repeat(dt[0], P, 1), np.repeat(A, P)[:, None] * np.ones(N),
                                 B[0], C[0], [L], np.repeat(D, P), None, h0.reshape(1, -1, N), on=False)
    np.testing.assert_allclose(f["y"], np.asarray(y, np.float64).reshape(L, -1), rtol=1e-9, atol=1e-9)
    np.testing.assert_allclose(f["final"], np.asarray(fin, np.float64).reshape(1, -1, N), rtol=1e-9, atol=1e-9)


@pytest.mark.parametrize("lens", [[4], [2, 0, 1, 3], [0]])
@pytest.mark.parametrize("gated,skip,act", [(True, True, "bias"), (False, False, "none"), (True, False, "clamp")])
def test_gradients(lens, gated, skip, act):
    rng, C, G, N, n, T = RNG(1), 4, 2, 3, len(lens), sum(lens)
    a = {"x": rng.standard_normal((T, C)), "dt": rng.uniform(0.1, 0.9, (T, C)) if act == "none" else
         rng.standard_normal((T, C)), "A": -rng.uniform(0.2, 3, (C, N)), "B": rng.standard_normal((T, G, N)),
         "C": rng.standard_normal((T, G, N)), "init": rng.standard_normal((n, C, N))}
    if gated:
        a["z"] = rng.standard_normal((T, C))
    if skip:
        a["D"] = rng.standard_normal(C)
    kw = {"on": False} if act == "none" else {"bias": rng.standard_normal(C)}
    if act == "clamp":
        kw["limit"] = (0.3, 1.0)
    if "bias" in kw:
        a["dt_bias"] = kw["bias"]
    dy, df = rng.standard_normal((T, C)), rng.standard_normal((n, C, N))

    def f():
        r = selective.selective_scan(a["x"], a["dt"], a["A"], a["B"], a["C"], lens, a.get("D"), a.get("z"), a["init"],
                                     **kw)
        return (r["y"] * dy).sum() + (r["final"] * df).sum()
    g, s = selective.selective_scan_backward(dy, a["x"], a["dt"], a["A"], a["B"], a["C"], lens, a.get("D"), a.get("z"),
                                             a["init"], df, **kw)
    for name in a:
        to = {"dt": "ddt", "dt_bias": "ddt_bias"}.get(name, "d" + name)
        differences(f, a, name, g[to])
        assert (np.abs(g[to]) <= s[to] * (1 + 1e-12)).all(), name


def test_step_sizes():
    d, slope = selective.step_sizes(np.array([-50.0, 0.0, 50.0]), limit=(0.01, 3.0))
    np.testing.assert_allclose(d, [0.01, np.log(2), 3.0])
    np.testing.assert_allclose(slope, [0.0, 0.5, 0.0])
    assert np.array_equal(block.softplus(0.0), np.log(2.0))
