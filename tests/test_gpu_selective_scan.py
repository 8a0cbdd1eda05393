"""The selective scan, its gradients and its single-token step against the fp64
oracle: state counts from one to 64, groups, lengths around the tiles, the saved
states and the items, empty sequences, activations, types, column ranges."""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import say
from oracle import selective
from selective_helpers import DTYPES, GRAD, OUT, STATE, Case, flat, make, rounded, up, within

pytestmark = pytest.mark.gpu

CASES = [
    # lens, dense, C, N, G, dtype, gated, skip, act, init, wide
    ([1], True, 8, 1, 1, "f32", False, False, "none", False, False),
    ([5], True, 24, 4, 1, "f32", True, True, "bias", True, False),
    ([16, 16], True, 16, 16, 1, "f32", False, True, "bias", True, False),
    ([33], False, 40, 16, 2, "bf16", True, True, "plain", False, True),
    ([130, 130], True, 136, 16, 1, "bf16", True, True, "bias", True, False),
    ([1, 700, 0, 63, 64, 65, 0], False, 72, 16, 1, "bf16", True, True, "bias", True, False),
    ([257, 3, 0, 129], False, 64, 11, 2, "f32", False, True, "clamp", True, True),
    ([200], True, 264, 8, 1, "f32", True, False, "bias", False, False),
    ([95], False, 104, 16, 8, "bf16", True, True, "bias", True, False),
    ([77, 77, 77], True, 32, 7, 4, "bf16", False, True, "none", True, False),
    ([150, 2], False, 48, 32, 1, "f32", True, True, "bias", True, False),
    ([90], True, 56, 27, 1, "bf16", True, True, "bias", True, True),
    ([131, 70], False, 24, 64, 1, "f32", True, True, "bias", True, False),
    ([0, 66, 1], False, 16, 50, 2, "bf16", True, True, "clamp", True, False),
    ([515], True, 8, 2, 1, "f32", True, True, "bias", True, False),
    ([0, 0], False, 16, 16, 1, "bf16", True, True, "bias", True, False),
    ([0, 0], True, 16, 16, 1, "f32", True, True, "bias", True, False),
    ([], False, 16, 16, 1, "f32", True, True, "bias", True, False),
    ([7 * k % 5 for k in range(1500)], False, 8, 16, 1, "bf16", True, True, "bias", True, False),
    ([2] * 700, True, 24, 3, 3, "f32", True, True, "bias", True, False),
]


def check_forward(c, v, kw, lens, dtype):
    ref = selective.selective_scan(v["x"], v["dt"], v["A"], v["B"], v["Cm"], lens, v["D"], v["z"], v["init"], **kw)
    y, final, states = ssd.selective_scan(*c.args, **c.kw, want_states=True)
    assert y.dtype == DTYPES[dtype] and y.shape == c.x.shape
    within(flat(y, ref["y"]), ref["y"], ref["y_s"], OUT, dtype, "y")
    within(final, ref["final"], ref["final_s"], STATE, "f32", "final state")
    other = "f32" if dtype == "bf16" else "bf16"
    y2, none = ssd.selective_scan(*c.args, **c.kw, y_dtype=DTYPES[other], want_final=False)
    assert none is None and y2.dtype == DTYPES[other]
    within(flat(y2, ref["y"]), ref["y"], ref["y_s"], OUT, other, "y in the other type")
    return states


NAMES = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinit")


def check_backward(got, ref, sc, dtype, lens, C):
    tokens = max([min(n, 65536) for n in lens] + [0])
    extra = {"dA": tokens + len(lens), "dD": tokens + len(lens), "ddt_bias": tokens + len(lens), "dB": 16 + C // 128,
             "dC": 16 + C // 128}
    for name, g in zip(NAMES, got):
        if name not in ref:
            assert g is None, name
            continue
        dt = dtype if name in ("dx", "ddt", "dB", "dC", "dz") else "f32"
        within(flat(g, ref[name]), ref[name], sc[name], GRAD + extra.get(name, 0), dt, name)


@pytest.mark.parametrize("lens,dense,C,N,G,dtype,gated,skip,act,init,wide", CASES)
def test_scan(lens, dense, C, N, G, dtype, gated, skip, act, init, wide):
    say("case: selective scan", lens, dense, C, N, G, dtype, gated, skip, act, init, wide)
    rng = np.random.default_rng(sum(lens) + C + N)
    v, kw = make(rng, lens, C, N, G, dtype, gated, skip, act, init)
    c = Case(v, kw, lens, dtype, dense, wide)
    states = check_forward(c, v, kw, lens, dtype)
    dy = rounded(rng, (sum(lens), C), dtype)
    for with_final in (True, False):
        df = rounded(rng, (len(lens), C, N), "f32") if with_final else None
        ref, sc = selective.selective_scan_backward(dy, v["x"], v["dt"], v["A"], v["B"], v["Cm"], lens, v["D"], v["z"],
                                                    v["init"], df, **kw)
        if "bias" not in kw:
            del ref["ddt_bias"]
        if v["D"] is None:
            del ref["dD"]
        got = ssd.selective_scan_backward(c.rows(dy), *c.args, states, dfinal_state=up(df), **c.kw)
        check_backward(got, ref, sc, dtype, lens, C)


@pytest.mark.parametrize("b,C,N,G,dtype,gated,skip,act", [
    (1, 8, 1, 1, "f32", False, False, "none"), (3, 40, 16, 1, "bf16", True, True, "bias"),
    (2, 64, 11, 2, "f32", True, True, "clamp"), (5, 24, 64, 1, "bf16", False, True, "plain"),
    (7, 136, 20, 1, "f32", True, False, "bias"), (0, 16, 16, 1, "bf16", True, True, "bias")])
def test_step(b, C, N, G, dtype, gated, skip, act):
    say("case: selective step", b, C, N, G, dtype, gated, skip, act)
    rng = np.random.default_rng(b + C + N)
    lens = [1] * b
    v, kw = make(rng, lens, C, N, G, dtype, gated, skip, act)
    ref = selective.selective_scan(v["x"], v["dt"], v["A"], v["B"], v["Cm"], lens, v["D"], v["z"], v["init"], **kw)
    for wide in (False, True):
        c = Case(v, kw, lens, dtype, False, wide)
        opts = {k: t for k, t in c.kw.items() if k not in ("init_state", "cu_seqlens")}
        state, out = c.init.clone(), torch.full_like(c.init, float("nan"))
        y = ssd.selective_scan_step(state, *c.args, state_out=out, **opts)
        assert torch.equal(state, c.init)
        within(y, ref["y"], ref["y_s"], OUT, dtype, "y")
        within(out, ref["final"], ref["final_s"], STATE, "f32", "state")
        y2 = ssd.selective_scan_step(state, *c.args, **opts)
        assert torch.equal(y2, y) and torch.equal(state, out)
