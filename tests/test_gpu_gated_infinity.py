"""An infinity in the gated recurrence: its own sequence stays infinite from
there on (a is positive, the input weight too), the others do not notice."""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import offsets, say, up
from test_gpu_gated_scan import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [np.inf, -np.inf])
@pytest.mark.parametrize("decay", [(-9.0, -3.5), (-9.0, 3.0)])
def test_infinity_stays(value, decay):
    """With decays of exp(-0.25) a token and more no run of rows forgets the state, so every later one is the
    infinity itself; where a run's factor underflows to 0 it may be no number, but it is never finite."""
    say("case: gated infinity", value, decay)
    lens = [150, 300, 1, 129]
    d = make(91, lens, 16, "f32", decay=decay)
    args = {k: up(d[k]) for k in ("x", "r", "i", "lam")}
    kw = dict(init_state=up(d["init"]), cu_seqlens=offsets(lens))
    clean, cfin = ssd.gated_scan(*args.values(), **kw)
    args["x"] = args["x"].clone()
    args["x"][200] = value
    y, fin = ssd.gated_scan(*args.values(), **kw)
    keep = np.r_[0:200, 450:sum(lens)]
    assert torch.equal(y[keep], clean[keep]) and torch.equal(fin[[0, 2, 3]], cfin[[0, 2, 3]])
    assert bool((y[200] == value).all())
    assert not torch.isfinite(y[200:450]).any() and not torch.isfinite(fin[1]).any()
    if decay[1] < -3:
        assert bool((y[200:450] == value).all()) and bool((fin[1] == value).all())
    state = up(d["init"])
    x = up(d["x"][:4])
    x[2] = value
    y = ssd.gated_scan_step(state, x, up(d["r"][:4]), up(d["i"][:4]), args["lam"])
    assert bool((y[2] == value).all()) and torch.isfinite(y[[0, 1, 3]]).all()
