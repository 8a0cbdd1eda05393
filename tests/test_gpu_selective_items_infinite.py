"""A state's way over the items a sequence is cut into: the factor exp(A S) of an item is
positive and finite however small or large fp32 makes it, so a state of 0 stays 0 and an
infinite one stays infinite over items, as token by token."""
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import say

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("N", [16, 5])
@pytest.mark.parametrize("packed", [False, True])
def test_infinity_stays(packed, N, sign):
    """Decays of exp(-2) a token: the factor of the 128 tokens of an item underflows, no single one does.  The last
    sequence's infinity is in its initial state."""
    say("case: selective scan, infinity over items", packed, N, sign)
    b, L, C = 3, 900, 16
    g = torch.Generator(device="cuda").manual_seed(N)
    x, dt, dy = (torch.rand(b, L, C, generator=g, device="cuda") + 0.5 for _ in range(3))
    B, Cm = (torch.rand(b, L, 1, N, generator=g, device="cuda") + 0.5 for _ in range(2))
    A = -(torch.rand(C, N, generator=g, device="cuda") + 1.0)
    init = torch.zeros(b, C, N, device="cuda")
    cu = torch.arange(0, b * L + 1, L, dtype=torch.int32, device="cuda") if packed else None

    def run(x, init, dy, df=None):
        rows = [t.flatten(0, 1) if packed else t for t in (x, dt, B, Cm, dy)]
        kw = dict(init_state=init, cu_seqlens=cu)
        args = (rows[0], rows[1], A, rows[2], rows[3])
        y, f, states = ssd.selective_scan(*args, want_states=True, **kw)
        got = ssd.selective_scan_backward(rows[4], *args, states, dfinal_state=df, **kw)
        return y.view(b, L, C), f, got[0].view(b, L, C), got[8]
    y0, f0, dx0, di0 = run(x, init, dy)
    bad = x.clone()
    bad[1, 10, 3] = sign * INF
    other = init.clone()
    other[2, 7] = sign * INF
    y, f, _, _ = run(bad, other, dy)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[1, 10:, 3] = hit[2, :, 7] = True
    assert torch.equal(y[~hit], y0[~hit]) and (y[hit] == sign * INF).all()
    ends = torch.zeros_like(f, dtype=torch.bool)
    ends[1, 3] = ends[2, 7] = True
    assert torch.equal(f[~ends], f0[~ends]) and (f[ends] == sign * INF).all()
    # the adjoint, from its other end
    bad = dy.clone()
    bad[1, L - 10, 3] = sign * INF
    df = torch.zeros_like(init)
    df[2, 7] = sign * INF
    _, _, dx, di = run(x, init, bad, df)
    _, _, dx0, di0 = run(x, init, dy, torch.zeros_like(init))
    hit = torch.zeros_like(dx, dtype=torch.bool)
    hit[1, :L - 9, 3] = hit[2, :, 7] = True
    assert torch.equal(dx[~hit], dx0[~hit]) and (dx[hit] == sign * INF).all()
    assert torch.equal(di[~ends], di0[~ends]) and (di[ends] == sign * INF).all()


def test_growth_of_nothing():
    """States that grow by exp(1) a token: an item's factor overflows, but there is nothing that it multiplies until
    the last tokens."""
    say("case: selective scan, growth of nothing")
    b, L, C, N = 2, 700, 16, 16
    x = torch.zeros(b, L, C, device="cuda")
    x[:, -3:] = 1.0
    dt = torch.ones_like(x)
    B = torch.ones(b, L, 1, N, device="cuda")
    A = torch.ones(C, N, device="cuda")
    y, f, states = ssd.selective_scan(x, dt, A, B, B, want_states=True)
    assert not y[:, :-3].any()
    e = torch.e
    want = torch.tensor([1.0, 1 + e, 1 + e + e * e], dtype=torch.float64, device="cuda")
    # each of three tokens: the exponential 2 u, the exponent's product and the sum 1 u each; the sum over 16 states 16
    assert ((y[:, -3:].double() - 16 * want[None, :, None]).abs() <= 32 * 2.0 ** -24 * 16 * want[None, :, None]).all()
    assert ((f.double() - want[2]).abs() <= 16 * 2.0 ** -24 * want[2]).all()
    # the same from the other end: gradients of outputs that are the first tokens'
    dy = torch.zeros_like(x)
    dy[:, :3] = 1.0
    got = ssd.selective_scan_backward(dy, x, dt, A, B, B, states)
    assert not got[0][:, 3:].any()
    assert ((got[0][:, :3].double() - 16 * want.flip(0)[None, :, None]).abs()
            <= 32 * 2.0 ** -24 * 16 * want.flip(0)[None, :, None]).all()
