"""The gated linear recurrence (gated_scan, its step and its gradients) against
the fp64 oracle: dense and packed batches, sequences of no and of one token and
across many tiles, both types, memories from none to thousands of tokens,
column ranges of wider tensors, saturated and infinite gate logits, NaN kept
inside its own sequence, rows behind the last sequence, other streams, captured
graphs, and a prefill continued by steps.

Error counts, in units of 2^-24 of the scale (sums of absolute values):
  sigmoid(v), |v| <= 6   exp2's argument 2|v|, exp2 2, add 1, reciprocal 2: <= 17
  log a                  softplus (4) and the factor 6 more: 23 of itself, so at most
                         23 |S| exp(-|S|) <= 9 in a product of a over any run
  the recurrence         a's rounding and one more a row of a run of rows: 16; b: 17 + 12 + 4
  a run's factor P       its sum, exp2 and their product with the state: 16 a run,
                         over the runs that the memory reaches
so a state is off by at most 64 + 16 runs, runs = min(L, memory) / 8 + 1.  A
gradient multiplies an adjoint (the same count) and a state and gates: twice
that and 64; dlam adds the roundings of its sum.
"""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from oracle import block
from block_helpers import DTYPES, down, in_wider, offsets, rounded, say, up, within

pytestmark = pytest.mark.gpu


def make(seed, lens, C, dtype, decay=(-7.0, 0.0), init=True):
    rng, T, n = np.random.default_rng(seed), sum(lens), len(lens)
    d = {k: rounded(rng, (T, C), dtype) for k in ("x", "r", "i", "dy")}
    d["lam"] = rng.uniform(*decay, C).astype(np.float32)
    d["init"] = rounded(rng, (n, C), "f32") if init else None
    d["dfinal"] = rounded(rng, (n, C), "f32") if init else None
    return d


def count(d, lens, rate=8.0):
    loga = block.gates(d["x"], d["r"], d["i"], d["lam"], rate)[0]
    if not loga.size:
        return 64
    memory = 1.0 / max(-np.expm1(loga.max()), 1e-9)
    return 64 + 16 * (min(max(lens), memory) / 8 + 1)


def check(d, lens, dtype, ydtype="f32", dense=False, wide=False, rate=8.0, extra=0, backward=True,
          floor=1e-30):
    """Forward and backward against the oracle; returns the GPU results."""
    T, C, n = sum(lens), d["x"].shape[1], len(lens)
    lead = (n, lens[0]) if dense else (T + extra,)

    def put(a, dt):
        if extra:
            a = np.concatenate([a, np.full((extra, C), np.nan, np.float32)])
        return in_wider(a, dt, lead) if wide else up(a, dt).view(lead + (C,))
    x, r, i = (put(d[k], dtype) for k in ("x", "r", "i"))
    lam, init, dfinal = up(d["lam"]), up(d["init"]), up(d["dfinal"])
    kw = dict(rate=rate, init_state=init, cu_seqlens=None if dense else offsets(lens))
    y0 = torch.full(lead + (C,), 7.0, dtype=DTYPES[ydtype], device="cuda")
    y, fin, states = ssd.gated_scan(x, r, i, lam, y=y0, want_states=True, **kw)
    yr, fr, scale = block.gated_scan(d["x"], d["r"], d["i"], d["lam"], lens, rate, d["init"])
    c = count(d, lens, rate)
    flat = y.view(-1, C)
    within(flat[:T], yr, scale, c, ydtype, "y", floor)
    assert bool((flat[T:] == 7.0).all()), "rows behind the last sequence"
    last = np.array([scale[hi - 1] if hi > lo else np.abs(fr[s]) for s, (lo, hi) in enumerate(block.bounds(lens))])
    within(fin, fr, last.reshape(n, C), c, "f32", "final_state", floor)
    y2, fin2 = ssd.gated_scan(x, r, i, lam, y_dtype=DTYPES[ydtype], **kw)
    assert torch.equal(y2.view(-1, C)[:T], flat[:T]) and torch.equal(fin2, fin), "the same call twice"
    if not backward:
        return y, fin
    dyq = torch.from_numpy(d["dy"]).to(DTYPES[ydtype]).float().numpy()
    dy = up(np.concatenate([dyq, np.full((extra, C), np.nan, np.float32)]), ydtype).view(lead + (C,))
    bk = dict(dfinal_state=dfinal, **kw)
    if wide:
        g = torch.full(lead + (3 * C,), 7.0, dtype=DTYPES[dtype], device="cuda")
        bk.update(zip(("dx", "dr", "di"), g.split(C, -1)))
    elif extra:
        bk.update({k: torch.full(lead + (C,), 7.0, dtype=DTYPES[dtype], device="cuda") for k in ("dx", "dr", "di")})
    got = dict(zip(("dx", "dr", "di", "dlam", "dinit"), ssd.gated_scan_backward(dy, x, r, i, lam, states, **bk)))
    ref, sc = block.gated_scan_backward(dyq, d["x"], d["r"], d["i"], d["lam"], lens, rate, d["init"], d["dfinal"])
    for k in ("dx", "dr", "di"):
        v = got[k].reshape(-1, C)
        within(v[:T], ref[k], sc[k], 2 * c + 64, dtype, k, floor)
        assert bool((v[T:] == 7.0).all()) or not extra, k + " behind the last sequence"
    within(got["dlam"], ref["dlam"], sc["dlam"], 2 * c + 128 + T / 128, "f32", "dlam", floor * T)
    within(got["dinit"], ref["dinit"], sc["dinit"], c, "f32", "dinit", floor)
    return y, fin


DENSE = [
    # b, L, C, dtype, ydtype, init, wide
    (1, 1, 8, "bf16", "bf16", True, False),
    (5, 1, 16, "f32", "f32", True, False),
    (1, 7, 64, "f32", "f32", False, False),
    (2, 128, 64, "bf16", "bf16", True, False),
    (3, 127, 72, "f32", "bf16", True, True),
    (2, 300, 136, "bf16", "f32", True, True),
    (1, 1024, 64, "bf16", "bf16", False, False),
    (1, 5003, 24, "f32", "f32", True, False),
    (37, 3, 200, "f32", "f32", True, False),
    (2, 2600, 40, "bf16", "bf16", True, True),
]


@pytest.mark.parametrize("b,L,C,dtype,ydtype,init,wide", DENSE)
def test_dense(b, L, C, dtype, ydtype, init, wide):
    say("case: gated dense", b, L, C, dtype, ydtype, init, wide)
    check(make(L + C, [L] * b, C, dtype, init=init), [L] * b, dtype, ydtype, dense=True, wide=wide)


PACKED = [
    # lens, C, dtype, rows behind
    ([5, 0, 1, 70, 2, 130, 0], 64, "bf16", 0),
    ([0, 0, 3], 16, "f32", 0),
    ([128, 128, 1, 127, 129], 136, "f32", 0),
    ([300, 3, 0, 129], 32, "bf16", 17),
    ([1] * 40, 8, "f32", 3),
    ([2500, 2049, 1], 72, "f32", 200),
    ([0, 0], 8, "f32", 0),
    ([0], 8, "bf16", 5),
    ([3001, 0, 5197], 1032, "bf16", 0),  # more than a round of workgroups, tiles no multiple of 8
]


@pytest.mark.parametrize("lens,C,dtype,extra", PACKED)
def test_packed(lens, C, dtype, extra):
    say("case: gated packed", lens, C, dtype, extra)
    check(make(C + sum(lens), lens, C, dtype), lens, dtype, dtype, extra=extra)


def test_memories_and_rates():
    """From a channel that forgets at once to one that keeps thousands of tokens."""
    say("case: gated memories")
    lens = [3000, 500]
    for decay, rate in [((-16.0, -12.0), 8.0), ((3.0, 40.0), 8.0), ((-100.0, -90.0), 8.0), ((-3.0, 0.0), 0.01)]:
        # below lam = -87 1 - a^2 is no normal number and counts as 0: what beta <= 2^-63 would have
        # weighed, up to 6 T of the values (at most 6) that meet it, is missing
        floor = 2.0 ** -63 * 6 * 6 * sum(lens) if decay[0] < -87 else 1e-30
        check(make(7, lens, 16, "f32", decay=decay), lens, "f32", rate=rate, floor=floor)


def test_saturated_and_infinite_logits():
    """sigmoid(r) of 0 keeps the state as it is and takes nothing in, of 1 decays
    by the full rate; infinities are their limits."""
    say("case: gated logits")
    for v in (90.0, 1e4, np.inf):
        lens = [40, 100]
        d = make(9, lens, 16, "f32", decay=(-3.0, 2.0))
        d["r"][::3] = -v
        d["r"][1::7] = v
        d["i"][::5] = -v
        d["i"][2::5] = v
        big = {k: np.clip(a, -1e4, 1e4) if k in "ri" else a for k, a in d.items()}  # the limits, in the oracle
        T, C = d["x"].shape
        # sigmoid(-90) = 2^-129.8 counts as 0 (its exponential overflows): what beta <= 2^-62 would have weighed,
        # up to 6 T of the values (at most 6) that meet it, is missing
        floor = 2.0 ** -62 * 6 * 6 * T
        kw = dict(init_state=up(d["init"]), cu_seqlens=offsets(lens))
        args = [up(d[k]) for k in ("x", "r", "i", "lam")]
        y, fin, states = ssd.gated_scan(*args, want_states=True, **kw)
        yr, fr, s = block.gated_scan(big["x"], big["r"], big["i"], d["lam"], lens, 8.0, d["init"])
        within(y, yr, s, 64 + 16 * 100, "f32", "y", floor)
        g = ssd.gated_scan_backward(up(d["dy"]), *args, states, dfinal_state=up(d["dfinal"]), **kw)
        ref, sc = block.gated_scan_backward(d["dy"], big["x"], big["r"], big["i"], d["lam"], lens, 8.0, d["init"],
                                            d["dfinal"])
        for k, v2 in zip(("dx", "dr", "di", "dlam", "dinit"), g):
            within(v2, ref[k], sc[k], 2 * (64 + 16 * 100) + 128, "f32", k, floor * T if k == "dlam" else floor)


@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_not_finite_stays_in_its_sequence(value):
    say("case: gated nan", value)
    lens = [150, 300, 1, 129]
    d = make(11, lens, 16, "f32", decay=(-9.0, 3.0))
    clean = check(d, lens, "f32")
    bad = {k: None if v is None else v.copy() for k, v in d.items()}
    bad["x"][200] = value   # inside the second sequence
    args = [up(bad[k]) for k in ("x", "r", "i", "lam")]
    kw = dict(init_state=up(d["init"]), cu_seqlens=offsets(lens))
    y, fin, states = ssd.gated_scan(*args, want_states=True, **kw)
    keep = np.r_[0:200, 450:sum(lens)]
    assert torch.equal(y[keep], clean[0][keep])
    assert torch.equal(fin[[0, 2, 3]], clean[1][[0, 2, 3]])
    assert not torch.isfinite(y[200:450]).any(1).any() or value == np.inf
    dy = d["dy"].copy()
    dy[300] = value
    good = ssd.gated_scan_backward(up(d["dy"]), *[up(d[k]) for k in ("x", "r", "i", "lam")],
                                   ssd.gated_scan(*[up(d[k]) for k in ("x", "r", "i", "lam")], want_states=True, **kw)[2],
                                   dfinal_state=up(d["dfinal"]), **kw)
    g = ssd.gated_scan_backward(up(dy), *args, states, dfinal_state=up(d["dfinal"]), **kw)
    out = np.r_[0:150, 450:sum(lens)]
    for k in range(3):
        assert torch.equal(g[k][out], good[k][out])
        assert torch.isfinite(g[k][out]).all()
    assert torch.equal(g[4][[0, 2, 3]], good[4][[0, 2, 3]])


def test_steps_continue_the_scan():
    say("case: gated steps")
    b, L, C, steps = 3, 130, 48, 9
    d = make(13, [L + steps] * b, C, "bf16")
    x, r, i = (up(d[k], "bf16").view(b, L + steps, C) for k in ("x", "r", "i"))
    lam = up(d["lam"])
    yr, fr, scale = block.gated_scan(d["x"], d["r"], d["i"], d["lam"], [L + steps] * b, 8.0, d["init"])
    _, state = ssd.gated_scan(*(v[:, :L].contiguous() for v in (x, r, i)), lam, init_state=up(d["init"]))
    c = count(d, [L + steps])
    yr, scale = yr.reshape(b, -1, C), scale.reshape(b, -1, C)
    for t in range(L, L + steps):
        before = state.clone()
        other = torch.empty_like(state)
        # the token's row of each sequence: rows L + steps apart
        y = ssd.gated_scan_step(state, x[:, t], r[:, t], i[:, t], lam, state_out=other, y_dtype=torch.float32)
        assert torch.equal(state, before)
        y2 = ssd.gated_scan_step(state, x[:, t], r[:, t], i[:, t], lam)
        assert torch.equal(state, other) and torch.equal(y2, y.to(torch.bfloat16))
        within(y, yr[:, t], scale[:, t], c + 8 * steps, "f32", "step %d" % t)
    within(state, fr, scale[:, -1], c + 8 * steps, "f32", "state")


def test_step_sizes():
    for b, C, dtype in [(1, 8, "f32"), (0, 8, "f32"), (7, 1000, "bf16"), (300, 24, "bf16")]:
        say("case: gated step", b, C, dtype)
        d = make(b + C, [1] * b, C, dtype)
        d["init"] = np.zeros((0, C), np.float32) if not b else d["init"]
        state = up(d["init"])
        y = ssd.gated_scan_step(state, *(up(d[k], dtype) for k in ("x", "r", "i")), up(d["lam"]))
        yr, fr, s = block.gated_scan(d["x"], d["r"], d["i"], d["lam"], [1] * b, 8.0, d["init"])
        within(y, yr, s, 64, dtype, "y")
        within(state, fr, s, 64, "f32", "state")


def test_other_stream_and_graph():
    """The call on a stream of its own, then captured and replayed on changing
    inputs with eager work between the replays."""
    say("case: gated graph")
    lens, C = [700, 0, 1300, 30], 72
    d = make(17, lens, C, "bf16")
    x, r, i, dy = (up(d[k], "bf16") for k in ("x", "r", "i", "dy"))
    lam, init, df, cu = up(d["lam"]), up(d["init"]), up(d["dfinal"]), offsets(lens)

    def both(x):
        y, fin, st = ssd.gated_scan(x, r, i, lam, init_state=init, cu_seqlens=cu, want_states=True)
        return (y, fin, *ssd.gated_scan_backward(dy, x, r, i, lam, st, init_state=init, dfinal_state=df, cu_seqlens=cu))
    want = both(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = both(x)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    xin = x.clone()
    with torch.cuda.stream(s):
        both(xin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(xin)
    for k in range(4):
        xk = x * (k + 1)
        xin.copy_(xk)
        want = both(xk)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), "replay %d" % k


def test_two_calls_at_once():
    """Passes of many tiles on two streams side by side, over and over, each the bits it gives alone."""
    say("case: gated two streams")
    C, args = 520, []
    for k in range(2):
        d = make(31 + k, [64] * 4, C, "bf16")
        x, r, i = (up(np.tile(d[n], (16 + 8 * k, 1)), "bf16").view(2, -1, C) for n in ("x", "r", "i"))
        args.append((x, r, i, up(d["lam"])))

    def both(a):
        y, fin, st = ssd.gated_scan(*a, want_states=True)
        return (y, fin, *ssd.gated_scan_backward(y, *a, st, dfinal_state=fin))
    want = [both(a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = [[], []]
    for _ in range(5):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(both(args[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(a, b) for run in got[k] for a, b in zip(run, want[k]))


def test_one_tile_of_very_many_channels():
    say("case: gated many channels")
    C, L = 66056, 5
    d = make(41, [L], C, "f32")
    cols = np.r_[0:64, 32000:32064, C - 72:C]
    args = [up(d[k]).view(1, L, C) for k in ("x", "r", "i")] + [up(d["lam"])]
    y, fin, st = ssd.gated_scan(*args, init_state=up(d["init"]), want_states=True)
    got = ssd.gated_scan_backward(up(d["dy"]).view(1, L, C), *args, st, init_state=up(d["init"]),
                                  dfinal_state=up(d["dfinal"]))
    part = {k: v[..., cols] for k, v in d.items()}
    yr, fr, scale = block.gated_scan(part["x"], part["r"], part["i"], part["lam"], [L], 8.0, part["init"])
    within(y[0][:, cols], yr, scale, 80, "f32", "y")
    ref, sc = block.gated_scan_backward(part["dy"], part["x"], part["r"], part["i"], part["lam"], [L], 8.0, part["init"],
                                        part["dfinal"])
    for k, v in zip(("dx", "dr", "di", "dlam", "dinit"), got):
        within(v.reshape(-1, C)[:, cols].reshape(ref[k].shape), ref[k], sc[k], 2 * 80 + 128, "f32", k)


def test_no_sequences_and_no_tokens():
    say("case: gated empty")
    lam = torch.zeros(16, device="cuda")
    for b, L in ((0, 7), (3, 0)):
        x = torch.zeros(b, L, 16, device="cuda")
        h = torch.randn(b, 16, device="cuda")
        y, fin, st = ssd.gated_scan(x, x, x, lam, init_state=h, want_states=True)
        assert y.shape == x.shape and torch.equal(fin, h) and st.shape == (0, 16)
        dx, _, _, dlam, dinit = ssd.gated_scan_backward(x, x, x, x, lam, st, init_state=h, dfinal_state=h)
        assert dx.shape == x.shape and not dlam.any() and torch.equal(dinit, h)
        assert not ssd.gated_scan(x, x, x, lam)[1].any()


def test_bad_offsets_stay_in_bounds():
    """Offsets that decrease, leave the stream or start late: no result is
    promised, but nothing outside the tensors is touched and the call ends."""
    C, T = 16, 400
    d = make(19, [T], C, "f32")
    x, r, i = (up(d[k]) for k in ("x", "r", "i"))
    for cu in ([0, 300, 100, 400], [0, 900, 1000, 400], [-50, 10, 20, 400], [37, 100, 200, 390], [0, -5, -9, 2 ** 31 - 1]):
        say("case: gated bad offsets", cu)
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kw = dict(init_state=up(d["init"]).expand(3, C).contiguous(), cu_seqlens=c)
        guard = torch.full((T + 2, C), 7.0, device="cuda")
        y, fin, st = ssd.gated_scan(x, r, i, up(d["lam"]), y=guard[1:-1], want_states=True, **kw)
        ssd.gated_scan_backward(up(d["dy"]), x, r, i, up(d["lam"]), st, dfinal_state=fin, **kw)
        torch.cuda.synchronize()
        assert bool((guard[[0, -1]] == 7.0).all())


def test_wide_addresses():
    """Elements past 2^31: the last rows of a stream of 2^31 + elements are read and written where they lie."""
    C, T = 16384, 131072 + 200
    say("case: gated wide", T, C)
    z = torch.zeros((T, C), dtype=torch.bfloat16, device="cuda")
    lens = [T - 200, 200]
    d = make(23, [200], C, "bf16")
    x, r, i = z, z.clone(), z.clone()
    for t, k in ((x, "x"), (r, "r"), (i, "i")):
        t[-200:] = up(d[k], "bf16")
    y, fin = ssd.gated_scan(x, r, i, up(d["lam"]), cu_seqlens=offsets(lens))
    cols = np.r_[0:8, C - 8:C]
    yr, fr, s = block.gated_scan(*(d[k][:, cols] for k in ("x", "r", "i")), d["lam"][cols], [200], 8.0)
    within(y[-200:][:, cols], yr, s, count(d, [200]), "bf16", "y")
    assert not y[:-200].any()
