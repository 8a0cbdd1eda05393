"""The selective scan where sequences are cut into many items, or none: long ones of
few channels, many channels at once, and packed ones of very different lengths;
against a token by token recurrence in float64 on the GPU, gradients by
differentiating it.

Tolerances: errors are bounded by c u of the scale (oracle/selective.py), here taken
from a run of the same recurrence on absolute values, which needs |v| = |dt A| below 2
so that (1 + |v|) is at most 3: every relative count of the short tests times 3.  A sum
over tokens adds one rounding a token."""
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from block_helpers import U, say

pytestmark = pytest.mark.gpu


def reference(x, dt, A, B, Cm, D, z, init, lens, positive=False):
    """y and the final states in float64; with `positive` of the absolute values, the magnitudes."""
    f = torch.abs if positive else (lambda v: v)
    step = torch.nn.functional.softplus(dt.double())
    x, B, Cm, D, init = (f(v.double()) for v in (x, B, Cm, D, init))
    a = torch.exp(step[..., None] * A.double())
    b = (step * x)[..., None] * B[:, :1]
    hs, ends = [], []
    at = 0
    for s, n in enumerate(lens):
        h = init[s]
        for t in range(at, at + n):
            h = a[t] * h + b[t]
            hs.append(h)
        ends.append(h)
        at += n
    p = (torch.stack(hs) * Cm[:, :1]).sum(-1) + D * x
    zz = z.double()
    gate = torch.nn.functional.silu(zz)
    return p * f(gate), torch.stack(ends)


@pytest.mark.parametrize("lens,dense,C,N,dtype", [
    ([4200], True, 16, 16, torch.float32),       # many items of the least length
    ([1100, 1100, 1100], True, 24, 8, torch.bfloat16),
    ([1, 2500, 0, 130, 64, 700], False, 40, 16, torch.float32),
    ([150], True, 32768, 4, torch.bfloat16),     # one item: 2048 waves
    ([70, 70], True, 16640, 3, torch.float32),
    ([130, 1, 90], False, 16640, 5, torch.bfloat16),
])
def test_against_float64(lens, dense, C, N, dtype):
    say("case: selective scan, items", lens, C, N, dtype)
    torch.manual_seed(sum(lens) + C)
    T, n = sum(lens), len(lens)

    def rnd(*s):
        return torch.randn(*s, device="cuda").clamp_(-4, 4)
    x, z, dy = (rnd(T, C).to(dtype) for _ in range(3))
    dt = (rnd(T, C) - 2).to(dtype)
    B, Cm = (rnd(T, 1, N).to(dtype) for _ in range(2))
    A = -torch.rand(C, N, device="cuda") * 0.7 - 0.01  # |dt A| < 2
    D, init, df = rnd(C), rnd(n, C, N), rnd(n, C, N)
    lead = (n, lens[0]) if dense else (T,)
    shaped = [v.view(lead + v.shape[1:]) for v in (x, dt, B, Cm, z, dy)]
    cu = None if dense else torch.tensor([sum(lens[:k]) for k in range(n + 1)], dtype=torch.int32, device="cuda")
    kw = dict(D=D, z=shaped[4], dt_softplus=True, init_state=init, cu_seqlens=cu)
    args = (shaped[0], shaped[1], A, shaped[2], shaped[3])
    y, final, states = ssd.selective_scan(*args, want_states=True, **kw)
    got = ssd.selective_scan_backward(shaped[5], *args, states, dfinal_state=df, **kw)

    leaves = [v.detach().double().requires_grad_() for v in (x, dt, A, B, Cm, D, z, init)]
    yr, fr = reference(*leaves[:3], *leaves[3:], lens)
    grads = torch.autograd.grad([yr, fr], leaves, [dy.double(), df.double()])
    with torch.no_grad():
        ys, fs = reference(x, dt, A, B, Cm, D, z, init, lens, True)

    def close(g, r, scale, c, name):
        g, r = g.detach().double().view(r.shape), r.detach()
        tol = c * U * scale + (2.0 ** -8 * r.abs() if g.dtype != torch.float32 and name in BF else 0)
        bad = ~((g - r).abs() <= tol + 1e-30)
        assert not bad.any(), "%s: %d of %d off, by up to %.3g of the tolerance" % (
            name, bad.sum(), bad.numel(), ((g - r).abs() / (tol + 1e-30)).max())
    BF = ("y", "dx", "ddt", "dB", "dC", "dz") if dtype == torch.bfloat16 else ()
    # a decay's error is carried along the tokens it lasts: the magnitude times the tokens of a memory,
    # bounded by those there are
    memory = 3 * 32
    close(y, yr, ys + ys.amax(0, keepdim=True), memory + 80, "y")
    close(final, fr, fs + fs.amax(), memory, "final")
    # gradients: of the size of the largest of a column or of all, whose terms they sum
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinit")
    order = (0, 1, 2, 3, 4, 5, 6, None, 7)
    for name, g, k in zip(names, got, order):
        if k is None:
            assert g is None
            continue
        r = grads[k]
        close(g, r, r.abs().amax().expand(r.shape), 3 * 128 + T, name)
