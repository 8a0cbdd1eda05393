"""Step sizes that the clamp cuts: their gradient is 0, whatever it is of, also infinite."""
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import DTYPES, offsets, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [16, 5])
def test_cut_steps(N, dtype):
    say("case: selective scan, cut steps", N, dtype)
    lens = [70, 3]
    T, C = sum(lens), 24
    g = torch.Generator(device="cuda").manual_seed(N)
    x, z, dy = (torch.rand(T, C, generator=g, device="cuda").add(0.25).to(DTYPES[dtype]) for _ in range(3))
    B, Cm = (torch.rand(T, 1, N, generator=g, device="cuda").add(0.25).to(DTYPES[dtype]) for _ in range(2))
    raw = torch.full((T, C), 5.0, device="cuda").to(DTYPES[dtype])  # softplus 5.007, cut to 0.5
    raw[:, 1::2] = -9.0  # 1.2e-4, cut to 0.1
    bias = torch.zeros(C, device="cuda")
    A = -torch.rand(C, N, generator=g, device="cuda")
    kw = dict(z=z, dt_softplus=True, dt_bias=bias, dt_limit=(0.1, 0.5), cu_seqlens=offsets(lens))
    _, _, states = ssd.selective_scan(x, raw, A, B, Cm, want_states=True, **kw)
    for at in (None, 3, 40):
        bad = dy.clone()
        if at is not None:
            bad[at] = float("inf")
        got = ssd.selective_scan_backward(bad, x, raw, A, B, Cm, states, **kw)
        assert not got[1].any() and not got[7].any(), (at, got[1], got[7])
        if at is not None:
            assert (got[0][:at + 1] == float("inf")).all()
