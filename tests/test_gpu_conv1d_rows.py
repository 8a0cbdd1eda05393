"""The conv1d gradients where a wave walks many batches of rows: blocks of 64 to
512 rows, dense and packed, with states on both sides.

Error counts, in units of 2^-24 of the scale: 64, as in the conv1d gradients' own
tests; a sum over tokens passes the rows of a wave, 3 waves, then the workgroups'
partial sums, blocks / 64 + 16.
"""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from mamba_ssd_chunked_02_amd import block_ops as ops
from oracle import block
from block_helpers import offsets, rounded, say, up, within

pytestmark = pytest.mark.gpu

CASES = [
    # lens, dense, C, K, dtype, dy's dtype, SiLU, rows of a wave
    ([270000, 270000], True, 8, 4, "bf16", "bf16", True, 128),
    ([1, 300000, 0, 2, 129999, 110001], False, 16, 3, "f32", "f32", True, 128),
    ([29000, 7, 993], False, 520, 4, "bf16", "f32", True, 16),
    ([70000], True, 264, 2, "bf16", "bf16", False, 32),
    ([35001, 0, 34999], False, 264, 4, "f32", "f32", False, 32),
]


@pytest.mark.parametrize("lens,dense,C,K,dtype,ydtype,silu,walk", CASES)
def test_long_walks(lens, dense, C, K, dtype, ydtype, silu, walk):
    say("case: conv backward of many rows", lens, C, K, dtype, ydtype)
    T, n = sum(lens), len(lens)
    torch.cuda.init()
    ops._lib()
    blocks = ops._conv_bytes(n, lens[0] if dense else T, C, K, not dense) // ((K + 1) * C * 4)
    assert -(-T // (4 * walk)) == blocks, "%d blocks" % blocks
    rng = np.random.default_rng(T + C)
    x, dy = rounded(rng, (T, C), dtype), rounded(rng, (T, C), ydtype)
    w, b = rounded(rng, (C, K), "f32", 0.5), rounded(rng, C, "f32")
    st, df = (rounded(rng, (n, K - 1, C), dtype) for _ in range(2))
    lead = (n, lens[0], C) if dense else (T, C)
    got = ssd.causal_conv1d_backward([up(dy, ydtype).view(lead)], up(x, dtype).view(lead), up(w), up(b),
                                     cu_seqlens=None if dense else offsets(lens), conv_state=up(st, dtype),
                                     dfinal_conv_state=up(df, dtype), activation=silu)
    ref, sc = block.causal_conv1d_backward(dy, x, w, b, lens, st, df, silu)
    sums = 64 + walk + 3 + blocks / 64 + 16
    within(got[0].view(T, C), ref["dx"], sc["dx"], 64, dtype, "dx")
    within(got[1], ref["dweight"], sc["dweight"], sums, "f32", "dweight")
    within(got[2], ref["dbias"], sc["dbias"], sums, "f32", "dbias")
    within(got[3], ref["dstate"], sc["dstate"], 64, dtype, "dstate")
