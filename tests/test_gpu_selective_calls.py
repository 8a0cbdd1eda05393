"""Calls of the selective scan as programs make them: captured and replayed, on two
streams at once, with a workspace and outputs of the caller's, column ranges of one
gradient tensor, rows behind the last sequence, offsets that are none, infinities,
sizes past 2^31 elements, and the same bits every time."""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import say
from selective_helpers import Case, make, rounded

pytestmark = pytest.mark.gpu


def a_case(lens, C, N, dtype="bf16", G=1, seed=0, dense=False, **kw):
    rng = np.random.default_rng(seed)
    v, act = make(rng, lens, C, N, G, dtype, **kw)
    c = Case(v, act, lens, dtype, dense)
    c.dy = c.rows(rounded(rng, (sum(lens), C), dtype))
    return c


def everything(c, **kw):
    y, final, states = ssd.selective_scan(*c.args, **c.kw, want_states=True)
    return (y, final, *ssd.selective_scan_backward(c.dy, *c.args, states, dfinal_state=final, **c.kw, **kw))


def same(a, b):
    return all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


def test_same_bits_again():
    say("case: selective scan twice")
    c = a_case([700, 0, 3, 1200], 136, 16)
    one = everything(c)
    for _ in range(3):
        assert same(one, everything(c))


def test_captured():
    say("case: selective scan graph")
    c = a_case([300, 1, 0, 260], 72, 16, "f32")
    x = c.x.clone()
    c.args = (x,) + c.args[1:]
    state, step_out = c.init[:1].clone(), torch.empty_like(c.init[:1])
    step = {k: v for k, v in c.kw.items() if k not in ("init_state", "cu_seqlens", "z")}

    def work():
        y = ssd.selective_scan_step(state, x[:1], c.dt[:1], c.A, c.B[:1], c.C[:1], state_out=step_out, **step)
        return (*everything(c), y, step_out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for k in range(4):
        x.copy_(c.x * (k + 1))
        want = [None if t is None else t.clone() for t in work()]
        torch.cuda.synchronize()
        for t in out:
            if t is not None and t is not step_out:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want), "replay %d" % k


def test_two_streams():
    """Two scans in flight, each with its own workspace from the binding."""
    say("case: selective scan streams")
    cs = [a_case([900, 40], 200, 16, seed=1), a_case([1300], 104, 8, seed=2)]
    want = [everything(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(everything(c))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))


def test_given_outputs_and_workspace():
    """Gradients as column ranges of wider tensors, next to what is left as it was; a workspace twice as large as
    needed and one too small, which is not used."""
    say("case: selective scan outputs")
    lens, C, N, G = [100, 0, 333], 56, 11, 2
    c = a_case(lens, C, N, "bf16", G)
    want = everything(c)
    T = sum(lens)
    nan = float("nan")
    wide = torch.full((T, 3 * C + 24), nan, dtype=torch.bfloat16, device="cuda")
    rows = torch.full((T, 2 * G * N + 5), nan, dtype=torch.bfloat16, device="cuda")
    dx, ddt, dz = (wide[:, 8 + k * C:8 + (k + 1) * C] for k in range(3))
    dB, dC = (rows[:, 3 + k * G * N:3 + (k + 1) * G * N].unflatten(-1, (G, N)) for k in range(2))
    for size in (1 << 26, 64):
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        y = torch.full_like(c.x, nan)
        final = torch.full_like(c.init, nan)
        got = ssd.selective_scan(*c.args, **c.kw, want_states=True, y=y, final_state=final, workspace=ws)
        assert got[0] is y and got[1] is final
        back = ssd.selective_scan_backward(c.dy, *c.args, got[2], dfinal_state=final, **c.kw, dx=dx, ddt=ddt, dz=dz, dB=dB,
                                           dC=dC, workspace=ws)
        assert same((y, final, *back), want)
    assert torch.isnan(wide[:, :8]).all() and torch.isnan(wide[:, 8 + 3 * C:]).all()
    assert torch.isnan(rows[:, :3]).all() and torch.isnan(rows[:, 3 + 2 * G * N:]).all()
    none = ssd.selective_scan_backward(c.dy, *c.args, got[2], dfinal_state=final, **c.kw, want_dinit=False)
    assert none[8] is None and same(none[:8], want[2:10])


def test_rows_behind_the_last_sequence():
    say("case: selective scan rows behind")
    lens = [70, 5, 130]
    c = a_case(lens, 40, 16, "f32")
    want = everything(c)
    T, more = sum(lens), 37

    def longer(t):
        return torch.cat([t, torch.full((more,) + tuple(t.shape[1:]), float("nan"), device="cuda", dtype=t.dtype)])
    args = (longer(c.x), longer(c.dt), c.A, longer(c.B), longer(c.C))
    kw = {**c.kw, "z": longer(c.z)}
    y = torch.full_like(args[0], 7.0)
    _, final, states = ssd.selective_scan(*args, **kw, want_states=True, y=y)
    outs = {k: torch.full_like(t, 7.0) for k, t in (("dx", args[0]), ("ddt", args[0]), ("dz", args[0]), ("dB", args[3]),
                                                    ("dC", args[3]))}
    back = ssd.selective_scan_backward(longer(c.dy), *args, states, dfinal_state=final, **kw, **outs)
    cut = [t[:T] if t is not None and t.shape[:1] == (T + more,) else t for t in back]
    assert same((y[:T], final, *cut), want)
    assert (y[T:] == 7).all() and all((t[T:] == 7).all() for t in outs.values())


def test_offsets_that_are_none():
    """Offsets that decrease or leave the rows: nothing outside the rows is touched, the call returns."""
    say("case: selective scan bad offsets")
    c = a_case([64, 64, 64], 24, 16, "f32")
    for bad in ([0, 200, 10, 192], [-5, 64, 128, 1000], [192, 128, 64, 0], [50, 60, 60, 70]):
        kw = {**c.kw, "cu_seqlens": torch.tensor(bad, dtype=torch.int32, device="cuda")}
        y, final, states = ssd.selective_scan(*c.args, **kw, want_states=True)
        ssd.selective_scan_backward(c.dy, *c.args, states, **kw)
        torch.cuda.synchronize()
        with pytest.raises(ssd.SsdError):
            ssd.selective_scan(*c.args, **kw, cu_seqlens_host=bad)
    ok = {**c.kw, "cu_seqlens_host": [0, 64, 128, 192]}
    assert torch.equal(ssd.selective_scan(*c.args, **ok)[0], ssd.selective_scan(*c.args, **c.kw)[0])


@pytest.mark.parametrize("N", [16, 5])
def test_not_finite(N):
    """NaN and infinity stay in their channel and behind their token; a decay rate of minus infinity forgets at once,
    also where a tile has rows without tokens; a step of 0 changes nothing."""
    say("case: selective scan not finite", N)
    lens = [61, 77]
    c = a_case(lens, 24, N, "f32", act="none")
    clean, clean_final = ssd.selective_scan(*c.args, **c.kw)
    x = c.x.clone()
    x[20, 3] = float("nan")
    x[70, 5] = float("inf")
    y, final = ssd.selective_scan(x, *c.args[1:], **c.kw)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[20:61, 3] = True
    hit[70:138, 5] = True
    assert torch.equal(y[~hit], clean[~hit])
    assert torch.isnan(y[20:61, 3]).all() and not torch.isfinite(y[70, 5])
    keep = torch.ones_like(final, dtype=torch.bool)
    keep[0, 3] = keep[1, 5] = False
    assert torch.equal(final[keep], clean_final[keep])
    A = c.A.clone()
    A[7] = -float("inf")
    y, final = ssd.selective_scan(c.x, c.dt, A, *c.args[3:], **c.kw)
    last = torch.tensor([60, 137], device="cuda")
    want = (c.dt * c.x)[last, 7, None] * c.B[last, 0]
    assert torch.equal(final[:, 7], want) and torch.isfinite(y).all()
    dt = c.dt.clone()
    dt[61:] = 0
    _, final = ssd.selective_scan(c.x, dt, A, *c.args[3:], **c.kw)
    assert torch.equal(final[1], c.init[1])


def test_past_2_31_elements():
    """Rows whose elements lie past 2^31 of x, y and the gradients, and a state past it."""
    say("case: selective scan wide")
    C, T, N = 16384, 140000, 1
    x = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    dt = torch.zeros_like(x)
    B = torch.ones(T, 1, N, dtype=torch.bfloat16, device="cuda")
    A = -torch.ones(C, N, device="cuda")
    lens = [T - 300, 300]
    cu = torch.tensor([0, T - 300, T], dtype=torch.int32, device="cuda")
    x[-300:] = torch.randn(300, C, device="cuda").bfloat16()
    dt[-300:] = (torch.rand(300, C, device="cuda") * 0.1).bfloat16()
    y, final, states = ssd.selective_scan(x, dt, A, B, B, cu_seqlens=cu, want_states=True)
    y2, final2, states2 = ssd.selective_scan(x[-300:].clone(), dt[-300:].clone(), A, B[-300:].clone(), B[-300:].clone(),
                                             cu_seqlens=torch.tensor([0, 300], dtype=torch.int32, device="cuda"),
                                             want_states=True)
    # the same tokens, cut into other items: one rounding a token and those of a carry
    tol = 400 * 2.0 ** -24 * y2.float().abs().max() + 2.0 ** -8 * y2.float().abs()
    assert ((y[-300:].float() - y2.float()).abs() <= 2 * tol).all() and not y[:-300].any()
    assert ((final[1] - final2[0]).abs() <= 400 * 2.0 ** -24 * final2.abs().max()).all() and not final[0].any()
    dy = torch.zeros_like(x)
    dy[-300:] = x[-300:]
    del y
    got = ssd.selective_scan_backward(dy, x, dt, A, B, B, states, cu_seqlens=cu)
    want = ssd.selective_scan_backward(dy[-300:].clone(), x[-300:].clone(), dt[-300:].clone(), A, B[-300:].clone(),
                                       B[-300:].clone(), states2,
                                       cu_seqlens=torch.tensor([0, 300], dtype=torch.int32, device="cuda"))
    for k in (0, 1, 3, 4):
        a, b = got[k][-300:].float(), want[k].float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 700 * 2.0 ** -24 * b.abs().max()).all(), k
    assert ((got[2] - want[2]).abs() <= 1000 * 2.0 ** -24 * want[2].abs().max()).all()
    del got, want, x, dt, dy
    # a step over more than 2^31 states
    b, C, N = 520, 65536, 64
    state = torch.zeros(b, C, N, device="cuda")
    state[-1] = 1.0
    xs = torch.ones(b, C, dtype=torch.bfloat16, device="cuda")
    Bs = torch.zeros(b, 1, N, dtype=torch.bfloat16, device="cuda")
    Cs = torch.ones_like(Bs)
    ys = ssd.selective_scan_step(state, xs, xs, torch.zeros(C, N, device="cuda"), Bs, Cs)
    assert (ys[-1] == 64).all() and not ys[:-1].any() and (state[-1] == 1).all() and not state[0].any()


def test_strided_steps():
    """A token's slice x[:, t] of a batch of long sequences: rows a sequence apart."""
    say("case: selective step strides")
    b, L, C, N = 3, 70, 40, 16
    c = a_case([L] * b, C, N, "bf16", dense=True)
    kw = {k: v for k, v in c.kw.items() if k not in ("init_state", "cu_seqlens", "z")}
    y, final = ssd.selective_scan(*c.args, **c.kw)
    state = c.init.clone()
    for t in range(L):
        got = ssd.selective_scan_step(state, c.x[:, t], c.dt[:, t], c.A, c.B[:, t], c.C[:, t], z=c.z[:, t], **kw)
        # y is rounded once from sums in another order
        tol = 2.0 ** -7 * y[:, t].float().abs() + 400 * 2.0 ** -24 * y.float().abs().max()
        assert ((got.float() - y[:, t].float()).abs() <= tol).all(), t
    assert ((state - final).abs() <= 400 * 2.0 ** -24 * final.abs().max()).all()


def test_most_channels():
    """2^20 channels of 64 states: their sums take more workgroups than one launch holds lanes for."""
    say("case: selective scan of 2^20 channels")
    C, N, L, some = 1 << 20, 64, 3, 1024
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dt, dy = (torch.randn(1, L, C, generator=g, device="cuda") for _ in range(3))
    B, Cm = (torch.randn(1, L, 1, N, generator=g, device="cuda") for _ in range(2))
    A = -torch.rand(C, N, generator=g, device="cuda") * 4
    bias, D = (torch.randn(C, generator=g, device="cuda") for _ in range(2))
    y, final, states = ssd.selective_scan(x, dt, A, B, Cm, D=D, dt_softplus=True, dt_bias=bias, want_states=True)
    got = ssd.selective_scan_backward(dy, x, dt, A, B, Cm, states, D=D, dt_softplus=True, dt_bias=bias)
    for at in (0, C // 2, C - some):
        s = slice(at, at + some)
        cut = [t[..., s].contiguous() for t in (dy, x, dt)]
        kw = dict(D=D[s].contiguous(), dt_softplus=True, dt_bias=bias[s].contiguous())
        y1, final1, st = ssd.selective_scan(cut[1], cut[2], A[s].contiguous(), B, Cm, want_states=True, **kw)
        want = ssd.selective_scan_backward(*cut, A[s].contiguous(), B, Cm, st, **kw)
        # a channel's values are the same operations in the same order wherever it stands
        assert torch.equal(y[..., s], y1) and torch.equal(final[:, s], final1), at
        for name, a, b in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias"), got, want):
            if name in ("dx", "ddt"):
                assert torch.equal(a[..., s], b), (name, at)
            elif name in ("dA", "dD", "dbias"):
                assert torch.equal(a[s], b), (name, at)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_of_the_other_type(dtype):
    """dy in fp32 or bf16, whatever x is: a bf16 value is the same number in both."""
    say("case: selective scan dy's type", dtype)
    c = a_case([131, 0, 66], 40, 16, dtype)
    *_, states = ssd.selective_scan(*c.args, **c.kw, want_states=True)
    dy = torch.randn(c.x.shape, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").bfloat16()
    one = ssd.selective_scan_backward(dy, *c.args, states, **c.kw)
    two = ssd.selective_scan_backward(dy.float(), *c.args, states, **c.kw)
    for a, b in zip(one, two):
        assert a is None and b is None or torch.equal(a, b)
