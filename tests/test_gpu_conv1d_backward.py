"""Gradients of the causal conv1d against the fp64 oracle: dense and packed
batches, sequences shorter than the window and over many blocks, states with
gradients on both sides, parts, widths, types, rows behind the last sequence,
graphs.

Error counts, in units of 2^-24 of the scale (which holds what an error of v
does to silu'): v K + 2, the sigmoid 17 and silu' 4 more, the K products of dx
and the final state's gradient: 64; the sums over tokens add the roundings of a
wave's rows, the waves and the workgroups: at most one a row.
"""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from oracle import block
from block_helpers import DTYPES, offsets, rounded, say, up, within

pytestmark = pytest.mark.gpu


def check(lens, C, K, dtype, ydtype, silu=True, bias=True, state=True, parts=None, dense=False, extra=0):
    rng, T, n = np.random.default_rng(sum(lens) + C), sum(lens), len(lens)
    x, dy = rounded(rng, (T, C), dtype), rounded(rng, (T, C), ydtype)
    w, b = rounded(rng, (C, K), "f32", 0.5), rounded(rng, C, "f32") if bias else None
    st = rounded(rng, (n, K - 1, C), dtype) if state else None
    df = rounded(rng, (n, K - 1, C), dtype) if state else None
    lead = (n, lens[0]) if dense else (T + extra,)

    def put(a, dt):
        a = np.concatenate([a, np.full((extra, a.shape[1]), np.nan, np.float32)])
        return up(a, dt).view(lead + (a.shape[1],))
    cuts = np.cumsum([0] + (parts or [C]))
    dys = [put(np.ascontiguousarray(dy[:, lo:hi]), ydtype) for lo, hi in zip(cuts, cuts[1:])]
    dx0 = torch.full(lead + (C,), 7.0, dtype=DTYPES[dtype], device="cuda")
    kw = dict(cu_seqlens=None if dense else offsets(lens), conv_state=up(st, dtype), dfinal_conv_state=up(df, dtype),
              activation=silu, want_dstate=True)
    dx, dw, db, ds = ssd.causal_conv1d_backward(dys, put(x, dtype), up(w), up(b), dx=dx0, **kw)
    ref, sc = block.causal_conv1d_backward(dy, x, w, b, lens, st, df, silu)
    within(dx.view(-1, C)[:T], ref["dx"], sc["dx"], 64, dtype, "dx")
    assert bool((dx.view(-1, C)[T:] == 7.0).all()), "rows behind the last sequence"
    within(dw, ref["dweight"], sc["dweight"], 64 + T, "f32", "dweight")
    if bias:
        within(db, ref["dbias"], sc["dbias"], 64 + T, "f32", "dbias")
    else:
        assert db is None
    within(ds, ref["dstate"], sc["dstate"], 64, dtype, "dstate")


DENSE = [
    # b, L, C, K, dtype, ydtype, silu, bias, state
    (2, 100, 64, 4, "bf16", "bf16", True, True, True),
    (3, 1, 8, 4, "f32", "f32", True, True, True),
    (1, 2, 24, 3, "f32", "f32", False, False, True),
    (2, 130, 520, 4, "f32", "bf16", True, True, False),
    (1, 200, 1040, 2, "bf16", "f32", True, True, True),
    (4, 64, 512, 4, "bf16", "bf16", False, True, True),
    (2, 2000, 264, 4, "bf16", "bf16", True, True, True),
]


@pytest.mark.parametrize("b,L,C,K,dtype,ydtype,silu,bias,state", DENSE)
def test_dense(b, L, C, K, dtype, ydtype, silu, bias, state):
    say("case: conv backward dense", b, L, C, K, dtype, ydtype, silu, bias, state)
    check([L] * b, C, K, dtype, ydtype, silu, bias, state, dense=True)


PACKED = [
    # lens, C, K, dtype, state, rows behind
    ([5, 0, 1, 70, 2, 130, 0], 64, 4, "bf16", True, 0),
    ([0, 0, 3], 16, 4, "f32", True, 0),
    ([64, 64, 1, 63, 65], 136, 4, "f32", False, 0),
    ([200, 3, 0, 129], 32, 3, "bf16", True, 9),
    ([1] * 50, 8, 2, "f32", True, 0),
    ([0], 8, 4, "f32", True, 6),
    ([0, 0], 8, 4, "bf16", True, 0),
    ([31, 1025, 2, 2, 500], 264, 4, "bf16", True, 33),
]


@pytest.mark.parametrize("lens,C,K,dtype,state,extra", PACKED)
def test_packed(lens, C, K, dtype, state, extra):
    say("case: conv backward packed", lens, C, K, dtype, state, extra)
    check(lens, C, K, dtype, dtype, state=state, extra=extra)


def test_parts():
    say("case: conv backward parts")
    check([77, 300], 288, 4, "bf16", "bf16", parts=[256, 16, 16])
    check([77], 288, 4, "f32", "f32", parts=[8, 280], dense=True)


def test_bad_offsets_stay_in_bounds():
    C, T, K = 16, 400, 4
    x, dy = torch.randn(T, C, device="cuda"), torch.randn(T, C, device="cuda")
    w = torch.randn(C, K, device="cuda")
    for cu in ([0, 300, 100, 400], [0, 900, 1000, 400], [-50, 10, 20, 400], [37, 100, 200, 390], [0, -5, -9, 2 ** 31 - 1]):
        say("case: conv backward bad offsets", cu)
        guard = torch.full((T + 2, C), 7.0, device="cuda")
        ssd.causal_conv1d_backward([dy], x, w, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                   conv_state=torch.randn(3, K - 1, C, device="cuda"), dx=guard[1:-1])
        torch.cuda.synchronize()
        assert bool((guard[[0, -1]] == 7.0).all())


def test_graph():
    say("case: conv backward graph")
    lens, C, K = [300, 0, 45, 700], 72, 4
    x, dy = (torch.randn(sum(lens), C, device="cuda").bfloat16() for _ in range(2))
    w, b, cu = torch.randn(C, K, device="cuda"), torch.randn(C, device="cuda"), offsets(lens)
    st = torch.randn(4, K - 1, C, device="cuda").bfloat16()

    def call(x):
        return ssd.causal_conv1d_backward([dy], x, w, b, cu_seqlens=cu, conv_state=st, dfinal_conv_state=st)
    xin = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(xin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(xin)
    for k in range(4):
        xin.copy_(x * (k + 1))
        want = call(x * (k + 1))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b2) for a, b2 in zip(out, want)), "replay %d" % k
