"""The states of a dense batch lie in front of other memory: whatever that holds
(NaN here), the last, partly filled tile of rows has nothing of it in any
result."""
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import say, up
from test_gpu_gated_scan import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,L", [(1, 1), (5, 1), (3, 7), (2, 127), (1, 130), (1, 4100), (3, 1001)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_states_in_front_of_other_memory(b, L, dtype):
    say("case: gated states in front of other memory", b, L, dtype)
    C = 72
    d = make(51, [L] * b, C, dtype)
    x, r, i, dy = (up(d[k], dtype).view(b, L, C) for k in ("x", "r", "i", "dy"))
    lam = up(d["lam"])

    def ahead(a):
        t = torch.full((b + 9, C), float("nan"), device="cuda")
        t[:b] = up(a)
        return t[:b]

    def run(place):
        init, df = place(d["init"]), place(d["dfinal"])
        y, fin, st = ssd.gated_scan(x, r, i, lam, init_state=init, want_states=True)
        return (y, fin, *ssd.gated_scan_backward(dy, x, r, i, lam, st, init_state=init, dfinal_state=df))
    for got, want in zip(run(ahead), run(up)):
        assert torch.isfinite(got).all() and torch.equal(got, want)
