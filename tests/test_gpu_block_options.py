"""The documented options of the block operators that change where a result goes
or what is left out, each against the plain call, bit by bit: workspaces given
(of the size asked for, larger, too small), offsets on the host too, results not
wanted, outputs given, rows of one to three leading dimensions, column ranges."""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from mamba_ssd_chunked_02_amd import block_ops as ops
from block_helpers import offsets, say, up
from test_gpu_gated_scan import make

pytestmark = pytest.mark.gpu


def same(got, want):
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert (a is None and b is None) or (a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b))


def workspaces(need):
    for n in (need, need + 4096, max(need - 1, 0), 0):
        yield torch.full((n,), 0xa5, dtype=torch.uint8, device="cuda")
    yield torch.full((need // 4 + 8,), float("nan"), device="cuda")


@pytest.mark.parametrize("lens", [[700, 0, 1300, 30], [90], [40, 41]])
def test_recurrence(lens):
    say("case: options of the recurrence", lens)
    C, n = 72, len(lens)
    d = make(101, lens, C, "bf16")
    x, r, i, dy = (up(d[k], "bf16") for k in ("x", "r", "i", "dy"))
    lam, init, df, cu = up(d["lam"]), up(d["init"]), up(d["dfinal"]), offsets(lens)
    kw = dict(init_state=init, cu_seqlens=cu)
    y, fin, st = want = ssd.gated_scan(x, r, i, lam, want_states=True, **kw)
    back = ssd.gated_scan_backward(dy, x, r, i, lam, st, dfinal_state=df, **kw)
    host = np.concatenate([[0], np.cumsum(lens)])
    for h in (host.tolist(), host.astype(np.int64), cu.cpu()):
        same(ssd.gated_scan(x, r, i, lam, want_states=True, cu_seqlens_host=h, **kw), want)
        same(ssd.gated_scan_backward(dy, x, r, i, lam, st, dfinal_state=df, cu_seqlens_host=h, **kw), back)
    for w in workspaces(ops._gated_bytes(n, sum(lens), C, True, 0)):
        same(ssd.gated_scan(x, r, i, lam, want_states=True, workspace=w, **kw), want)
    for w in workspaces(ops._gated_bytes(n, sum(lens), C, True, 1)):
        same(ssd.gated_scan_backward(dy, x, r, i, lam, st, dfinal_state=df, workspace=w, **kw), back)
    y2, none = ssd.gated_scan(x, r, i, lam, want_final=False, **kw)
    assert none is None and torch.equal(y2, y)
    given = torch.empty_like(fin), torch.empty_like(y)
    y2, f2 = ssd.gated_scan(x, r, i, lam, want_final=False, final_state=given[0], y=given[1], **kw)
    assert f2 is given[0] and y2 is given[1] and torch.equal(f2, fin) and torch.equal(y2, y)
    got = ssd.gated_scan_backward(dy, x, r, i, lam, st, dfinal_state=df, want_dinit=False, **kw)
    same(got, (*back[:4], None))
    dl, di = torch.empty_like(lam), torch.empty_like(init)
    got = ssd.gated_scan_backward(dy, x, r, i, lam, st, dfinal_state=df, want_dinit=False, dlam=dl, dinit_state=di, **kw)
    assert got[3] is dl and got[4] is di
    same(got, back)
    # no initial state and no gradient of the final one: zeros
    zero = torch.zeros_like(init)
    same(ssd.gated_scan(x, r, i, lam, cu_seqlens=cu), ssd.gated_scan(x, r, i, lam, cu_seqlens=cu, init_state=zero))
    st0 = ssd.gated_scan(x, r, i, lam, cu_seqlens=cu, want_states=True)[2]
    same(ssd.gated_scan_backward(dy, x, r, i, lam, st0, cu_seqlens=cu),
         ssd.gated_scan_backward(dy, x, r, i, lam, st0, cu_seqlens=cu, init_state=zero, dfinal_state=zero))


def test_step():
    say("case: options of the step")
    d = make(102, [1] * 7, 40, "bf16")
    x, r, i = (up(d[k], "bf16") for k in ("x", "r", "i"))
    lam, state = up(d["lam"]), up(d["init"])
    a = state.clone()
    y = ssd.gated_scan_step(a, x, r, i, lam)
    b, out = torch.empty_like(state), torch.empty_like(y)
    assert ssd.gated_scan_step(state, x, r, i, lam, state_out=b, y=out) is out
    assert torch.equal(out, y) and torch.equal(a, b) and torch.equal(state, up(d["init"]))
    y32 = torch.empty(7, 40, device="cuda")
    assert ssd.gated_scan_step(state, x, r, i, lam, state_out=b, y=y32) is y32 and torch.equal(y32.bfloat16(), y)


@pytest.mark.parametrize("lead", [(), (5,), (3, 7), (2, 3, 4)])
@pytest.mark.parametrize("rdtype", [torch.bfloat16, torch.float32])
def test_residual_norm(lead, rdtype):
    say("case: options of the residual norm", lead, rdtype)
    D = 136
    gen = torch.Generator(device="cuda").manual_seed(103)

    def n(*shape, dt=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda").to(dt)
    x, dy = (n(*lead, D, dt=torch.bfloat16) for _ in range(2))
    res, dout = (n(*lead, D, dt=rdtype) for _ in range(2))
    w, s = n(D), n(D)
    want = ssd.add_rms_norm(x, res, w, scale=s, want_rstd=True)
    flat = ssd.add_rms_norm(x.reshape(-1, D), res.reshape(-1, D), w, scale=s, want_rstd=True)
    same([v.reshape(f.shape) for v, f in zip(want, flat)], flat)
    given = [torch.empty_like(x), torch.empty_like(res)]
    got = ssd.add_rms_norm(x, res, w, scale=s, y=given[0], residual_out=given[1])
    assert got[0] is given[0] and got[1] is given[1]
    same(got, want[:2])
    y, out, rstd = want
    kw = dict(dresidual_out=dout, x=x, scale=s)
    back = ssd.add_rms_norm_backward(dy, out, w, rstd, **kw)
    for ws in workspaces(ops._norm_bytes(x.numel() // D, D, 1)):
        same(ssd.add_rms_norm_backward(dy, out, w, rstd, workspace=ws, **kw), back)
    dx, dres = torch.empty_like(x), torch.empty_like(res)
    got = ssd.add_rms_norm_backward(dy, out, w, rstd, dx=dx, dresidual=dres, **kw)
    assert got[0] is dx and got[1] is dres
    same(got, back)
    # no scale: both gradients written where both are given
    one = ssd.add_rms_norm_backward(dy, out, w, rstd, dresidual_out=dout)
    two = ssd.add_rms_norm_backward(dy, out, w, rstd, dresidual_out=dout, dx=dx, dresidual=dres)
    assert two[0] is dx and two[1] is dres and (one[0] is one[1]) == (rdtype == torch.bfloat16)
    same(two, one)
    only = torch.empty_like(res)
    got = ssd.add_rms_norm_backward(dy, out, w, rstd, dresidual_out=dout, dresidual=only)
    assert got[1] is only
    same(got, one)


@pytest.mark.parametrize("lead", [(), (5,), (3, 7), (2, 3, 4)])
@pytest.mark.parametrize("groups,first", [(1, False), (2, True)])
def test_gated_norm(lead, groups, first):
    say("case: options of the gated norm", lead, groups, first)
    D = 144
    gen = torch.Generator(device="cuda").manual_seed(104)
    both = torch.randn(*lead, 3 * D, generator=gen, device="cuda").bfloat16()
    x, z, dy = both.split(D, -1)  # column ranges
    dy = dy.contiguous()
    w = torch.randn(D, generator=gen, device="cuda")
    kw = dict(groups=groups, norm_before_gate=first)
    want = ssd.gated_rms_norm(x.contiguous(), z.contiguous(), w, want_rstd=True, **kw)
    same(ssd.gated_rms_norm(x, z, w, want_rstd=True, **kw), want)
    y = torch.empty_like(want[0])
    assert ssd.gated_rms_norm(x, z, w, y=y, **kw) is y and torch.equal(y, want[0])
    back = ssd.gated_rms_norm_backward(dy, x.contiguous(), z.contiguous(), w, want[1], **kw)
    d = torch.full_like(both, 7.0)
    dx, dz, rest = d.split(D, -1)
    got = ssd.gated_rms_norm_backward(dy, x, z, w, want[1], dx=dx, dz=dz, **kw)
    assert got[0] is dx and got[1] is dz and bool((rest == 7.0).all())
    same(got, back)
    for ws in workspaces(ops._norm_bytes(dy.numel() // D, D, groups)):
        same(ssd.gated_rms_norm_backward(dy, x, z, w, want[1], workspace=ws, **kw), back)


@pytest.mark.parametrize("lens", [[300, 0, 45, 700], [5]])
def test_conv1d(lens):
    say("case: options of the conv1d gradients", lens)
    C, K, T, n = 72, 4, sum(lens), len(lens)
    gen = torch.Generator(device="cuda").manual_seed(105)
    x, dy = (torch.randn(T, C, generator=gen, device="cuda").bfloat16() for _ in range(2))
    w, b = torch.randn(C, K, generator=gen, device="cuda"), torch.randn(C, generator=gen, device="cuda")
    st = torch.randn(n, K - 1, C, generator=gen, device="cuda").bfloat16()
    kw = dict(cu_seqlens=offsets(lens), conv_state=st, dfinal_conv_state=st)
    want = ssd.causal_conv1d_backward([dy], x, w, b, **kw)
    for h in (np.concatenate([[0], np.cumsum(lens)]).tolist(), kw["cu_seqlens"].cpu()):
        same(ssd.causal_conv1d_backward((dy,), x, w, b, cu_seqlens_host=h, **kw), want)
    for ws in workspaces(ops._conv_bytes(n, T, C, K, True)):
        same(ssd.causal_conv1d_backward([dy], x, w, b, workspace=ws, **kw), want)
    same(ssd.causal_conv1d_backward([dy], x, w, b, want_dstate=False, **kw), (*want[:3], None))
    same(ssd.causal_conv1d_backward([dy], x, w, torch.zeros_like(b), **kw)[:2],
         ssd.causal_conv1d_backward([dy], x, w, **kw)[:2])
    zero = torch.zeros_like(st)
    cu = kw["cu_seqlens"]
    same(ssd.causal_conv1d_backward([dy], x, w, b, cu_seqlens=cu, want_dstate=True),
         ssd.causal_conv1d_backward([dy], x, w, b, cu_seqlens=cu, conv_state=zero, dfinal_conv_state=zero))
    dx = torch.empty_like(x)
    assert ssd.causal_conv1d_backward([dy], x, w, b, dx=dx, **kw)[0] is dx and torch.equal(dx, want[0])


def test_refusals_on_the_gpu():
    """What the binding refuses of GPU tensors, with its reason."""
    x = torch.zeros(2, 5, 16, device="cuda")
    lam, st = torch.zeros(16, device="cuda"), torch.zeros(1, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    rows = torch.zeros(3, 16, device="cuda")
    for f in (lambda: ssd.gated_scan(x, x[:, :4], x, lam), lambda: ssd.gated_scan(x[0], x[0], x[0], lam),
              lambda: ssd.gated_scan(x, x, x, lam[:8]), lambda: ssd.gated_scan(x, x, x, lam, init_state=st),
              lambda: ssd.gated_scan(x, x, x, lam.cpu()), lambda: ssd.gated_scan(x, x, x, lam, cu_seqlens_host=[0, 10]),
              lambda: ssd.gated_scan(x, x, x, lam, workspace=torch.empty(0, dtype=torch.uint8)),
              lambda: ssd.gated_scan(x, x, x.transpose(0, 1).contiguous().transpose(0, 1), lam),
              lambda: ssd.gated_scan_backward(x, x, x, x, lam, st[:, :8]),
              lambda: ssd.gated_scan_step(st, x, x, x, lam),
              lambda: ssd.add_rms_norm(rows, rows[:2], w), lambda: ssd.add_rms_norm(rows[:, ::2], rows, w),
              lambda: ssd.add_rms_norm_backward(rows, rows, w, rows[:, 0].contiguous(), scale=w),
              lambda: ssd.gated_rms_norm(rows, rows, w[:8]),
              lambda: ssd.causal_conv1d_backward([], rows, torch.zeros(16, 4, device="cuda")),
              lambda: ssd.causal_conv1d_backward([x] * 4, x, torch.zeros(16, 4, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            f()
    for f in (lambda: ssd.gated_scan(x.half(), x.half(), x.half(), lam), lambda: ssd.gated_scan(x, x.bfloat16(), x, lam),
              lambda: ssd.gated_scan(x, x, x, lam.double()), lambda: ssd.add_rms_norm(rows.half(), rows.half(), w),
              lambda: ssd.gated_rms_norm(rows, rows, w, y=torch.empty(3, 16, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            f()
    for f in (lambda: ssd.gated_scan(x, x, x, lam, rate=-1.0), lambda: ssd.gated_scan(x, x, x, lam, y=x),
              lambda: ssd.gated_scan(x[..., :12], x[..., :12], x[..., :12], lam[:12]),
              lambda: ssd.gated_scan(x.bfloat16()[..., 4:12], x.bfloat16()[..., 4:12], x.bfloat16()[..., 4:12], lam[:8]),
              lambda: ssd.add_rms_norm(rows, rows.bfloat16(), w), lambda: ssd.add_rms_norm(rows, rows, w, eps=-1.0),
              lambda: ssd.add_rms_norm(rows, rows.clone(), w, y=rows, residual_out=rows),
              lambda: ssd.gated_rms_norm(rows, rows, w, groups=3), lambda: ssd.gated_rms_norm(rows, rows, w, groups=0)):
        with pytest.raises(ssd.SsdError):
            f()


@pytest.mark.parametrize("groups", [2 ** 32 + 1, 2 ** 40 + 2, -(2 ** 32) + 1])
def test_groups_of_more_than_32_bits(groups):
    """Not taken for what their low 32 bits say."""
    x, w = torch.zeros(3, 16, device="cuda"), torch.ones(16, device="cuda")
    with pytest.raises(ValueError):
        ssd.gated_rms_norm(x, x, w, groups=groups)
    with pytest.raises(ValueError):
        ssd.gated_rms_norm_backward(x, x, x, w, torch.zeros(3, 1, device="cuda"), groups=groups)
