"""The fp64 oracle of the block operators (oracle.block) against itself: its
gradients against central differences of its forward pass, its recurrence
against the closed form at constant gates, its conv1d against oracle.conv."""
import numpy as np
import pytest

from oracle import block, conv

RNG = np.random.default_rng


def differences(f, args, name, grad, step=1e-5):
    """Central differences of the scalar f in args[name], entry by entry."""
    v = args[name]
    got = np.zeros_like(v)
    for at in np.ndindex(v.shape):
        keep = v[at]
        v[at] = keep + step
        hi = f()
        v[at] = keep - step
        lo = f()
        v[at] = keep
        got[at] = (hi - lo) / (2 * step)
    # the differences' own error: step^2 times a third derivative, and 2^-52 of the sum over 2 step
    np.testing.assert_allclose(grad, got, rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("lens", [[5], [3, 0, 1, 4], [0], [1, 1]])
def test_gated_scan_gradients(lens):
    rng, C, n, T = RNG(1), 3, len(lens), sum(lens)
    a = {k: rng.standard_normal((T, C)) for k in ("x", "r", "i")}
    a |= {"lam": rng.standard_normal(C) - 2, "init": rng.standard_normal((n, C))}
    dy, df = rng.standard_normal((T, C)), rng.standard_normal((n, C))

    def f():
        y, fin, _ = block.gated_scan(a["x"], a["r"], a["i"], a["lam"], lens, 2.0, a["init"])
        return (y * dy).sum() + (fin * df).sum()
    g, s = block.gated_scan_backward(dy, a["x"], a["r"], a["i"], a["lam"], lens, 2.0, a["init"], df)
    for name in a:
        differences(f, a, name, g["d" + name])
        assert (np.abs(g["d" + name]) <= s["d" + name] * (1 + 1e-12)).all(), name


def test_gated_scan_closed_form():
    """Constant gates: h_t = a^t h_0 + b (1 - a^t) / (1 - a)."""
    L, C = 50, 4
    lam = np.linspace(-6, 1, C)
    one = np.ones((L, C))
    y, fin, _ = block.gated_scan(3 * one, 0 * one, 0 * one, lam, [L], 8.0, np.full((1, C), 2.0))
    a = np.exp(-8.0 * np.log1p(np.exp(lam)) * 0.5)
    t = np.arange(1, L + 1)[:, None]
    b = np.sqrt(1 - a * a) * 0.5 * 3
    np.testing.assert_allclose(y, a ** t * 2 + b * (1 - a ** t) / (1 - a), rtol=1e-10)
    assert np.array_equal(fin[0], y[-1])


@pytest.mark.parametrize("scaled", [False, True])
def test_add_rms_norm_gradients(scaled):
    rng, rows, D = RNG(2), 3, 8
    a = {"x": rng.standard_normal((rows, D)), "residual": rng.standard_normal((rows, D)),
         "weight": rng.standard_normal(D)}
    if scaled:
        a["scale"] = rng.standard_normal(D)
    dy, do = rng.standard_normal((rows, D)), rng.standard_normal((rows, D))

    def f():
        y, out, _ = block.add_rms_norm(a["x"], a["residual"], a["weight"], a.get("scale"))
        return (y * dy).sum() + (out * do).sum()
    _, out, rstd = block.add_rms_norm(a["x"], a["residual"], a["weight"], a.get("scale"))
    g, s = block.add_rms_norm_backward(dy, out, a["weight"], rstd, do, a["x"], a.get("scale"))
    for name in a:
        differences(f, a, name, g["d" + name])
        assert (np.abs(g["d" + name]) <= s["d" + name] * (1 + 1e-12)).all(), name


@pytest.mark.parametrize("groups,first", [(1, False), (2, False), (1, True), (4, True)])
def test_gated_rms_norm_gradients(groups, first):
    rng, rows, D = RNG(3), 3, 8
    a = {"x": rng.standard_normal((rows, D)), "z": rng.standard_normal((rows, D)), "weight": rng.standard_normal(D)}
    dy = rng.standard_normal((rows, D))

    def f():
        return (block.gated_rms_norm(a["x"], a["z"], a["weight"], groups, 1e-3, first)[0] * dy).sum()
    g, s = block.gated_rms_norm_backward(dy, a["x"], a["z"], a["weight"], groups, 1e-3, first)
    for name in a:
        differences(f, a, name, g["d" + name])
        assert (np.abs(g["d" + name]) <= s["d" + name] * (1 + 1e-12)).all(), name


@pytest.mark.parametrize("lens,K,silu", [([5], 4, True), ([1, 0, 2, 3], 4, True), ([2, 4], 2, False), ([3, 1], 3, True)])
def test_conv1d_gradients(lens, K, silu):
    rng, C, n, T = RNG(4), 2, len(lens), sum(lens)
    a = {"x": rng.standard_normal((T, C)), "weight": rng.standard_normal((C, K)), "bias": rng.standard_normal(C),
         "state": rng.standard_normal((n, K - 1, C))}
    dy, df = rng.standard_normal((T, C)), rng.standard_normal((n, K - 1, C))
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)

    def f():
        y, fin = conv.causal_conv1d_batch(a["x"], a["weight"], a["bias"], a["state"], cu_seqlens=cu, activation=silu)
        return (y * dy).sum() + (fin * df).sum()
    g, s = block.causal_conv1d_backward(dy, a["x"], a["weight"], a["bias"], lens, a["state"], df, silu)
    for name in a:
        differences(f, a, name, g["d" + name])
        assert (np.abs(g["d" + name]) <= s["d" + name] * (1 + 1e-12)).all(), name
