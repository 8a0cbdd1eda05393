"""The selective scan without D: nothing is added to y, not 0 times an infinite x."""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import offsets, say, up

pytestmark = pytest.mark.gpu
INF = float("inf")

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
def test_no_skip(dtype, gated):
    """Without D nothing is added to y: an infinite x gives the infinity of its states, and an infinite gradient of y
    that of its adjoint."""
    say("case: selective scan, no skip", dtype, gated)
    rng = np.random.default_rng(3)
    T, C, N = 70, 16, 16
    x, B, Cm, z, dy = (up(rng.uniform(0.25, 1.0, s).astype(np.float32), dtype)
                       for s in ((T, C), (T, 1, N), (T, 1, N), (T, C), (T, C)))
    z = z if gated else None
    dt = up(rng.uniform(0.01, 0.1, (T, C)).astype(np.float32), dtype)
    A = -torch.ones(C, N, device="cuda")
    x = x.clone()
    dy = dy.clone()
    x[40, 3] = INF
    dy[50, 9] = INF
    cu = offsets([T])
    y, f, states = ssd.selective_scan(x, dt, A, B, Cm, z=z, cu_seqlens=cu, want_states=True)
    assert (y[40:, 3] == INF).all() and (f[0, 3] == INF).all()
    rest = [c for c in range(C) if c != 3]
    assert torch.isfinite(y[:, rest]).all() and torch.isfinite(y[:40]).all()
    got = ssd.selective_scan_backward(dy, x, dt, A, B, Cm, states, z=z, cu_seqlens=cu)
    assert (got[0][:51, 9] == INF).all()
    dx = got[0].clone()
    dx[:51, 9] = 0
    assert torch.isfinite(dx).all()
    if gated:
        assert (got[6][40:, 3] == INF).all() and torch.isfinite(got[6][:40]).all()
    state = torch.zeros(1, C, N, device="cuda")
    kw = dict(z=None if z is None else z[40:41])
    ys = ssd.selective_scan_step(state, x[40:41], dt[40:41], A, B[40:41], Cm[40:41], **kw)
    assert ys[0, 3] == INF and torch.isfinite(ys[0, rest]).all()


def test_no_skip_at_a_step_of_zero():
    """A step of 0 leaves the state as it is and adds nothing to y."""
    say("case: selective scan, a step of zero")
    T, C, N = 9, 8, 4
    x = torch.ones(1, T, C, device="cuda")
    dt = torch.zeros_like(x)
    B = torch.ones(1, T, 1, N, device="cuda")
    A = -torch.ones(C, N, device="cuda")
    init = torch.ones(1, C, N, device="cuda")
    y, f = ssd.selective_scan(x, dt, A, B, B, init_state=init)
    assert (y == N).all() and torch.equal(f, init)
