"""Decay rates that are not finite."""
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import offsets, say

pytestmark = pytest.mark.gpu
INF = float("inf")

@pytest.mark.parametrize("N", [16, 5])
def test_rate_of_plus_infinity(N):
    """exp(dt times infinity) is an infinity, and a positive state with it, also where the last tile has rows without
    tokens; a step of 0 leaves the state as it is."""
    say("case: selective scan, a rate of plus infinity", N)
    C = 16
    for lens in ([61, 3], [64, 130]):
        T = sum(lens)
        x, dt = torch.ones(T, C, device="cuda"), torch.full((T, C), 0.5, device="cuda")
        B = torch.ones(T, 1, N, device="cuda")
        A = -torch.ones(C, N, device="cuda")
        init = torch.ones(2, C, N, device="cuda")
        cu = offsets(lens)
        y0, f0 = ssd.selective_scan(x, dt, A, B, B, init_state=init, cu_seqlens=cu)
        A[3] = INF
        y, f = ssd.selective_scan(x, dt, A, B, B, init_state=init, cu_seqlens=cu)
        rest = [c for c in range(C) if c != 3]
        assert (y[:, 3] == INF).all() and (f[:, 3] == INF).all(), lens
        assert torch.equal(y[:, rest], y0[:, rest]) and torch.equal(f[:, rest], f0[:, rest])
        _, f = ssd.selective_scan(x, torch.zeros_like(dt), A, B, B, init_state=init, cu_seqlens=cu)
        assert torch.equal(f, init), lens
    state = init.clone()
    y = ssd.selective_scan_step(state, x[:2], dt[:2], A, B[:2], B[:2])
    assert (y[:, 3] == INF).all() and (state[:, 3] == INF).all() and torch.isfinite(state[:, rest]).all()
