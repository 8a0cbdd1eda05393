"""Sequences of many items, forward and backward, against the fp64 oracle with the scale of
every single element, as the short cases are (selective_helpers): what an item hands on
is checked where it arrives.

An item's factor exp(A S) is off by its exponent's 16 and the sum's roundings, one a token
of a lane's quarter of an item and two more, of |A S|, which the scale holds as (1 + |v|)
a token: STATE of each token covers 16 + 32 + 2 of their sum."""
import numpy as np
import pytest

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import say, up
from oracle import selective
from selective_helpers import Case, make, rounded
from test_gpu_selective_scan import check_backward, check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,dense,C,N,G,dtype,a_scale", [
    ([2600], True, 16, 16, 1, "f32", 1.0),
    ([2600], True, 16, 16, 1, "f32", 0.01),  # states that last over many items
    ([1, 1900, 0, 129, 640], False, 24, 11, 3, "f32", 0.05),
    ([1500, 1500], True, 40, 16, 1, "bf16", 0.02),
    ([2000], False, 8, 64, 1, "f32", 0.02),
    ([2000], False, 8, 3, 1, "bf16", 0.02),
])
def test_many_items(lens, dense, C, N, G, dtype, a_scale):
    say("case: selective scan, many items", lens, dense, C, N, G, dtype, a_scale)
    rng = np.random.default_rng(sum(lens) + C + N)
    v, kw = make(rng, lens, C, N, G, dtype, a_scale=a_scale)
    c = Case(v, kw, lens, dtype, dense)
    states = check_forward(c, v, kw, lens, dtype)
    dy, df = rounded(rng, (sum(lens), C), dtype), rounded(rng, (len(lens), C, N), "f32")
    ref, sc = selective.selective_scan_backward(dy, v["x"], v["dt"], v["A"], v["B"], v["Cm"], lens, v["D"], v["z"],
                                                v["init"], df, **kw)
    got = ssd.selective_scan_backward(c.rows(dy), *c.args, states, dfinal_state=up(df), **c.kw)
    check_backward(got, ref, sc, dtype, lens, C)
