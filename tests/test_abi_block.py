"""Host-side checks of the block operators' entry points: every refusal comes
back as its status before any launch (addresses that are never read stand in
for device pointers), and the binding refuses tensors off the GPU."""
import ctypes
import re

import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from mamba_ssd_chunked_02_amd import block_ops as ops
from test_abi_host import (E_ALIGN, E_DTYPE, E_NULL, E_SEQ, E_SHAPE, E_VALUE, E_WS, FAKE, HEADER, conv_outs,
                           conv_shape)

E_UNSUPPORTED = -8
BIG = 1 << 40  # workspace bytes


@pytest.fixture(scope="module")
def lib():
    return ops._lib()


def at(k):
    return FAKE + 4096 * (k + 1)


def gated_shape(**kw):
    s = ops._GatedShape()
    for k, v in {**dict(batch=2, seqlen=100, channels=64, dtype=1, ydtype=1, rate=8.0), **kw}.items():
        setattr(s, k, v)
    return s


FORWARD = ["x", "r", "i", "lam", "init", "y", "final", "states"]
BACKWARD = ["dy", "dfinal", "x", "r", "i", "lam", "init", "states", "dx", "dr", "di", "dlam", "dinit"]
STEP = ["state", "state_out", "x", "r", "i", "lam", "y"]


def call(f, names, sh, ws=True, size=BIG, **kw):
    p = {n: at(k) for k, n in enumerate(names)}
    p.update(kw)
    tail = ([at(40), size] if ws is True else [ws, size] if ws is not False else []) + [None]
    return f(*[p[n] for n in names], None if sh is None else ctypes.byref(sh), *tail)


def test_gated_refusals(lib):
    fwd = lambda sh=None, **kw: call(lib.ssd_gated_scan, FORWARD, gated_shape() if sh is None else sh, **kw)  # noqa: E731
    bwd = lambda sh=None, **kw: call(lib.ssd_gated_scan_backward, BACKWARD, gated_shape() if sh is None else sh, **kw)  # noqa: E731
    step = lambda sh=None, **kw: call(lib.ssd_gated_scan_step, STEP, gated_shape() if sh is None else sh, ws=False, **kw)  # noqa: E731
    assert call(lib.ssd_gated_scan, FORWARD, None) == E_NULL
    assert call(lib.ssd_gated_scan_backward, BACKWARD, None) == E_NULL
    assert call(lib.ssd_gated_scan_step, STEP, None, ws=False) == E_NULL
    for f in (fwd, bwd, step):
        assert f(gated_shape(dtype=2)) == E_DTYPE
        assert f(gated_shape(ydtype=-1)) == E_DTYPE
        assert f(gated_shape(reserved=1)) == E_SHAPE
        for c in (0, 4, 12, 2 ** 20 + 8, -8):
            assert f(gated_shape(channels=c)) == E_SHAPE, c
        for b in (-1, 2 ** 24 + 1):
            assert f(gated_shape(batch=b)) == E_SHAPE
        for rate in (0.0, -1.0, float("inf"), float("nan")):
            assert f(gated_shape(rate=rate)) == E_VALUE, rate
        for name in ("x_stride", "r_stride", "i_stride", "dx_stride", "dr_stride", "di_stride"):
            for v in (-64, 8, 56, 68):
                assert f(gated_shape(**{name: v})) == E_SHAPE, (name, v)
        for name in ("x", "r", "i", "lam"):
            assert f(**{name: None}) == E_NULL, name
            assert f(**{name: at(30) + 8}) == E_ALIGN, name
    for f in (fwd, bwd):
        assert f(gated_shape(seqlen=-1)) == E_SHAPE
        assert f(gated_shape(batch=2 ** 20, seqlen=2 ** 12)) == E_SHAPE
        assert f(ws=None) == E_WS
        assert f(size=16) == E_WS
        assert f(ws=at(40) + 8) == E_ALIGN
        host = (ctypes.c_int32 * 3)(0, 60, 40)
        sh = gated_shape(cu_seqlens=at(41), cu_seqlens_host=ctypes.addressof(host))
        assert f(sh) == E_SEQ
        host[:] = [1, 60, 100]
        assert f(sh) == E_SEQ
        host[:] = [0, 60, 101]
        assert f(sh) == E_SEQ
        assert f(gated_shape(cu_seqlens_host=ctypes.addressof(host))) == E_SHAPE
        assert f(gated_shape(batch=0, cu_seqlens=at(41))) == E_SHAPE
    assert fwd(y=at(0)) == E_SHAPE and fwd(final=at(4)) == E_SHAPE and fwd(states=at(6)) == E_SHAPE
    assert fwd(y=None) == E_NULL and fwd(y=at(30) + 8) == E_ALIGN
    for name in ("dy", "states", "dx", "dr", "di", "dlam"):
        assert bwd(**{name: None}) == E_NULL, name
    for name, other in (("dx", 2), ("dr", 0), ("di", 9), ("dlam", 5), ("dinit", 1)):
        assert bwd(**{name: at(other)}) == E_SHAPE, name
    for name in ("state", "state_out", "y"):
        assert step(**{name: None}) == E_NULL, name
    assert step(y=at(0)) == E_SHAPE and step(state_out=at(2)) == E_SHAPE
    n = ctypes.c_size_t(0)
    assert lib.ssd_gated_scan_workspace_size(ctypes.byref(gated_shape()), 2, ctypes.byref(n)) == E_VALUE
    assert lib.ssd_gated_scan_workspace_size(ctypes.byref(gated_shape()), 0, None) == E_NULL
    assert lib.ssd_gated_scan_workspace_size(ctypes.byref(gated_shape()), 0, ctypes.byref(n)) == 0 and n.value > 0
    assert fwd(size=n.value - 1) == E_WS


def norm_shape(**kw):
    s = ops._NormShape()
    for k, v in {**dict(rows=4, columns=64, groups=1, dtype=1, dtype2=1, eps=1e-5), **kw}.items():
        setattr(s, k, v)
    return s


def test_norm_refusals(lib):
    res = ["x", "residual", "weight", "scale", "y", "out", "rstd"]
    resb = ["dy", "dout", "out", "weight", "rstd", "x", "scale", "dx", "dresidual", "dweight", "dscale"]
    gate = ["x", "z", "weight", "y", "rstd"]
    gateb = ["dy", "x", "z", "weight", "rstd", "dx", "dz", "dweight"]
    every = [(lib.ssd_add_rms_norm, res, False), (lib.ssd_add_rms_norm_backward, resb, True),
             (lib.ssd_gated_rms_norm, gate, False), (lib.ssd_gated_rms_norm_backward, gateb, True)]
    optional = {"scale", "dscale", "dout", "dresidual"}
    for f, names, ws in every:
        gated = "z" in names
        go = lambda sh=None, **kw: call(f, names, norm_shape() if sh is None else sh, **{"ws": ws, **kw})  # noqa: E731
        assert call(f, names, None, ws=ws) == E_NULL
        assert go(norm_shape(dtype=3)) == E_DTYPE and go(norm_shape(dtype2=-1)) == E_DTYPE
        assert go(norm_shape(reserved=1)) == E_SHAPE
        for eps in (-1e-6, float("nan"), float("inf")):
            assert go(norm_shape(eps=eps)) == E_VALUE
        for c in (0, -8, 4, 12):
            assert go(norm_shape(columns=c)) == E_SHAPE, c
        assert go(norm_shape(columns=16392)) == E_UNSUPPORTED
        assert go(norm_shape(rows=-1)) == E_SHAPE and go(norm_shape(rows=2 ** 31)) == E_SHAPE
        assert go(norm_shape(rows=2 ** 30, columns=16384)) == E_SHAPE
        assert go(norm_shape(dtype=0, dtype2=1)) == E_UNSUPPORTED
        for g in (0, -1, 1025) + (() if gated else (2,)):
            assert go(norm_shape(groups=g)) == E_SHAPE, g
        assert go(norm_shape(norm_before_gate=2 if gated else 1)) == E_VALUE
        if gated:
            assert go(norm_shape(groups=3)) == E_SHAPE
            for v in (-64, 8, 68):
                for name in ("x_stride", "z_stride", "dx_stride", "dz_stride"):
                    assert go(norm_shape(**{name: v})) == E_SHAPE
        else:
            assert go(norm_shape(x_stride=64)) == E_SHAPE
        for k, name in enumerate(names):
            if not (name in optional or name == "rstd" and not ws):
                assert go(**{name: None}) == E_NULL, name
            assert go(**{name: at(30) + 4}) == E_ALIGN, name
        if ws:
            assert go(size=8) == E_WS and go(ws=None) == E_WS
            assert go(dx=at(0)) == E_SHAPE and go(dweight=at(names.index("dx"))) == E_SHAPE
        else:
            assert go(y=at(2)) == E_SHAPE and go(rstd=at(names.index("y"))) == E_SHAPE
    assert call(lib.ssd_add_rms_norm_backward, resb, norm_shape(), scale=None) == E_SHAPE  # dscale without scale
    assert call(lib.ssd_add_rms_norm, res, norm_shape(), ws=False, out=at(0)) == E_SHAPE
    assert call(lib.ssd_add_rms_norm_backward, resb, norm_shape(), dx=at(8)) == E_SHAPE  # dx is dresidual
    assert call(lib.ssd_add_rms_norm_backward, resb, norm_shape(dtype2=0), dx=at(1)) == E_SHAPE  # dout of another type
    n = ctypes.c_size_t(0)
    assert lib.ssd_norm_backward_workspace_size(ctypes.byref(norm_shape()), ctypes.byref(n)) == 0 and n.value >= 2 * 64 * 4


def test_conv_backward_refusals(lib):
    names = ["x", "weight", "bias", "state", "dstate_out", "dx", "dweight", "dbias", "dstate_in"]

    def go(sh=None, out=None, **kw):
        return call(lambda *a: lib.ssd_causal_conv1d_backward(ctypes.byref(conv_outs() if out is None else out), *a),
                    names, conv_shape() if sh is None else sh, **kw)
    assert lib.ssd_causal_conv1d_backward(None, *[at(k) for k in range(9)], ctypes.byref(conv_shape()), at(40), BIG,
                                          None) == E_NULL
    assert call(lambda *a: lib.ssd_causal_conv1d_backward(ctypes.byref(conv_outs()), *a), names, None) == E_NULL
    for kw, e in [(dict(dtype=2), E_DTYPE), (dict(ydtype=5), E_DTYPE), (dict(activation=2), E_VALUE),
                  (dict(reserved=1), E_SHAPE), (dict(width=1), E_SHAPE), (dict(width=5), E_SHAPE),
                  (dict(channels=12), E_SHAPE), (dict(batch=-1), E_SHAPE), (dict(seqlen=-1), E_SHAPE)]:
        assert go(conv_shape(**kw)) == e, kw
    for parts in ((32, 24), (60, 4)):
        assert go(out=conv_outs(parts)) == E_SHAPE
    o = conv_outs()
    o.nparts = 4
    assert go(out=o) == E_SHAPE
    o = conv_outs((32, 32))
    o.out[1] = None
    assert go(out=o) == E_NULL
    o = conv_outs()
    o.out[0] = at(30) + 8
    assert go(out=o) == E_ALIGN
    for name in ("x", "weight", "dx", "dweight"):
        assert go(**{name: None}) == E_NULL, name
    for k, name in enumerate(names):
        assert go(**{name: at(30) + 4}) == E_ALIGN, name
    for name in ("dx", "dweight", "dbias", "dstate_in"):
        assert go(**{name: at(0)}) == E_SHAPE, name
    assert go(size=64) == E_WS and go(ws=None) == E_WS
    host = (ctypes.c_int32 * 3)(0, 60, 40)
    assert go(conv_shape(cu_seqlens=at(41), cu_seqlens_host=ctypes.addressof(host))) == E_SEQ
    assert go(conv_shape(cu_seqlens_host=ctypes.addressof(host))) == E_SHAPE
    assert go(conv_shape(batch=0, cu_seqlens=at(41))) == E_SHAPE


def test_binding_constants_and_refusals():
    m = re.search(r"#define SSD_GATED_STATE_ROWS (\d+)", open(HEADER).read())
    assert m and int(m.group(1)) == ops.GATED_STATE_ROWS
    x, lam = torch.zeros(1, 4, 8), torch.zeros(8)
    with pytest.raises(ValueError):
        ssd.gated_scan(x, x, x, lam)
    with pytest.raises(ValueError):
        ssd.add_rms_norm(x, x, lam)
    with pytest.raises(ValueError):
        ssd.gated_rms_norm(x, x, lam)
    with pytest.raises(ValueError):
        ssd.causal_conv1d_backward([x], x, torch.zeros(8, 4))


def test_row_strides():
    """The distance of the rows, and tensors that have none."""
    w = torch.zeros(6, 5, 40)
    assert ops._row_stride(w, "x") == 0  # dense
    assert ops._row_stride(w[:, :, 8:24], "x") == 40
    assert ops._row_stride(w[:, 2], "x") == 200
    assert ops._row_stride(w[:1, :1], "x") == 0
    assert ops._row_stride(w[:, :1], "x") == 200
    assert ops._row_stride(w[:0], "x") == 0
    for bad in (w.transpose(0, 1), w[:, :3], w.transpose(1, 2), w[..., ::2], w[:1].expand(6, 5, 40)):
        with pytest.raises(ValueError):
            ops._row_stride(bad, "x")
