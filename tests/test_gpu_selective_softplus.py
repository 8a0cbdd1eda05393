"""The selective scan's softplus over its whole range."""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import U, down, offsets, say, up

pytestmark = pytest.mark.gpu

def raw_values():
    rng = np.random.default_rng(7)
    v = np.concatenate([rng.uniform(-87.0, 40.0, 1 << 15), rng.uniform(-2.0, 2.0, 1 << 14),
                        rng.uniform(-15.0, -1.0, 1 << 14), -2.0 ** rng.uniform(-30, 0, 1 << 13),
                        2.0 ** rng.uniform(-30, 0, 1 << 13)])
    return v.astype(np.float32)


def test_softplus():
    """With x, B and C of 1 and A of 0 a first token's state is its step size: softplus within 4 units of 2^-24,
    which the bounds of the other tests count."""
    say("case: selective scan, softplus")
    v = raw_values()
    C = 1 << 10
    raw = up(v.reshape(-1, C))
    n = raw.shape[0]
    one, ones = torch.ones_like(raw), torch.ones(n, 1, 1, device="cuda")
    A = torch.zeros(C, 1, device="cuda")
    want = np.maximum(v.astype(np.float64), 0) + np.log1p(np.exp(-np.abs(v.astype(np.float64))))
    y, f = ssd.selective_scan(one, raw, A, ones, ones, dt_softplus=True, cu_seqlens=offsets([1] * n))
    state = torch.zeros(n, C, 1, device="cuda")
    y2 = ssd.selective_scan_step(state, one, raw, A, ones, ones, dt_softplus=True)
    for got in (y, f, y2, state):
        off = np.abs(down(got).reshape(-1) - want) / (U * want)
        worst = int(off.argmax())
        assert off.max() <= 4.0, "softplus(%r) off by %.2f units" % (v[worst], off[worst])
