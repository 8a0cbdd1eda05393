"""Elements past 2^31: the gradients of the recurrence, the norms and the conv1d
read and write the last rows of tensors of 2^31 + elements where they lie.  The
rows before hold zeros, which leave nothing in a sum.  Error counts as in the
operators' own tests."""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from oracle import block
from block_helpers import offsets, rounded, say, up, within
from test_gpu_gated_scan import count, make

pytestmark = pytest.mark.gpu

C, TAIL = 16384, 200
T = 131072 + TAIL
COLS = np.r_[0:8, 8184:8200, C - 8:C]


def zeros_but(tail, dtype="bf16"):
    t = torch.zeros((T, C), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    t[-TAIL:] = up(tail, dtype)
    return t


def tail(t):
    assert not t[:-TAIL].any()
    return t[-TAIL:][:, COLS]


def test_recurrence():
    say("case: gated gradients, wide")
    d = make(81, [TAIL], C, "bf16")
    x, r, i, dy = (zeros_but(d[k]) for k in ("x", "r", "i", "dy"))
    lam, cu = up(d["lam"]), offsets([T - TAIL, TAIL])
    init, df = (torch.cat([torch.zeros(1, C, device="cuda"), up(d[k])]) for k in ("init", "dfinal"))
    _, _, states = ssd.gated_scan(x, r, i, lam, init_state=init, cu_seqlens=cu, want_states=True)
    got = ssd.gated_scan_backward(dy, x, r, i, lam, states, init_state=init, dfinal_state=df, cu_seqlens=cu)
    p = {k: v[..., COLS] for k, v in d.items()}
    c = count(p, [TAIL])
    ref, sc = block.gated_scan_backward(p["dy"], p["x"], p["r"], p["i"], p["lam"], [TAIL], 8.0, p["init"], p["dfinal"])
    for name, g in zip(("dx", "dr", "di"), got):
        within(tail(g), ref[name], sc[name], 2 * c + 64, "bf16", name)
    within(got[3][COLS], ref["dlam"], sc["dlam"], 2 * c + 128 + TAIL, "f32", "dlam")
    within(got[4][1:, COLS], ref["dinit"], sc["dinit"], c, "f32", "dinit")


def test_residual_norm():
    say("case: residual norm, wide")
    rng = np.random.default_rng(82)
    x, res, dy, dout = (rounded(rng, (TAIL, C), "bf16") for _ in range(4))
    w, s = rounded(rng, C, "f32"), rounded(rng, C, "f32")
    gx, gw, gs = zeros_but(x), up(w), up(s)
    y, out, rstd = ssd.add_rms_norm(gx, zeros_but(res), gw, scale=gs, want_rstd=True)
    yr, ur, rr = block.add_rms_norm(x, res, w, s)
    mag = np.abs(res) + np.abs(s * x)
    ymag = (mag + mag.max(-1, keepdims=True)) * rr[:, None] * np.abs(w)
    within(tail(y), yr[:, COLS], ymag[:, COLS], 64, "bf16", "y")
    within(tail(out), ur[:, COLS], mag[:, COLS], 2, "bf16", "out")
    got = ssd.add_rms_norm_backward(zeros_but(dy), out, gw, rstd, dresidual_out=zeros_but(dout), x=gx, scale=gs)
    ref, sc = block.add_rms_norm_backward(dy, out[-TAIL:].double().cpu().numpy(), w, rstd[-TAIL:].double().cpu().numpy(),
                                          dout, x, s)
    for name, g in zip(("dx", "dresidual"), got):
        within(tail(g), ref[name][:, COLS], sc[name][:, COLS], 128, "bf16", name)
    for name, g in zip(("dweight", "dscale"), got[2:]):
        within(g, ref[name], sc[name], 128 + TAIL, "f32", name)


def test_gated_norm():
    say("case: gated norm, wide")
    rng = np.random.default_rng(83)
    x, z, dy = (rounded(rng, (TAIL, C), "bf16") for _ in range(3))
    w = rounded(rng, C, "f32")
    gx, gz, gw = zeros_but(x), zeros_but(z), up(w)
    y, rstd = ssd.gated_rms_norm(gx, gz, gw, groups=4, want_rstd=True)
    yr, _ = block.gated_rms_norm(x, z, w, 4)
    within(tail(y), yr[:, COLS], np.abs(yr)[:, COLS], 64 + 23, "bf16", "y")
    got = ssd.gated_rms_norm_backward(zeros_but(dy), gx, gz, gw, rstd, groups=4)
    ref, sc = block.gated_rms_norm_backward(dy, x, z, w, 4)
    for name, g in zip(("dx", "dz"), got):
        within(tail(g), ref[name][:, COLS], sc[name][:, COLS], 128, "bf16", name)
    within(got[2], ref["dweight"], sc["dweight"], 128 + TAIL, "f32", "dweight")


def test_conv1d():
    say("case: conv backward, wide")
    rng, K = np.random.default_rng(84), 4
    x, dy = (rounded(rng, (TAIL, C), "bf16") for _ in range(2))
    w = rounded(rng, (C, K), "f32", 0.5)
    st, df = (rounded(rng, (1, K - 1, C), "bf16") for _ in range(2))
    gst, gdf = (torch.cat([torch.zeros(1, K - 1, C, device="cuda").bfloat16(), up(v, "bf16")]) for v in (st, df))
    got = ssd.causal_conv1d_backward([zeros_but(dy)], zeros_but(x), up(w), cu_seqlens=offsets([T - TAIL, TAIL]),
                                     conv_state=gst, dfinal_conv_state=gdf)
    ref, sc = block.causal_conv1d_backward(dy[:, COLS], x[:, COLS], w[COLS], None, [TAIL], st[..., COLS], df[..., COLS])
    within(tail(got[0]), ref["dx"], sc["dx"], 64, "bf16", "dx")
    within(got[1][COLS], ref["dweight"], sc["dweight"], 64 + TAIL, "f32", "dweight")
    within(got[3][1:][..., COLS], ref["dstate"], sc["dstate"], 64, "bf16", "dstate")
