"""Host-side checks of the selective scan's entry points: every refusal comes back
as its status before any launch, and the binding refuses what it should."""
import ctypes
import re

import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from mamba_ssd_chunked_02_amd import SsdError, _DtAct
from mamba_ssd_chunked_02_amd import block_ops as ops
from mamba_ssd_chunked_02_amd import selective_ops as sel
from test_abi_block import at, call
from test_abi_host import E_ALIGN, E_DTYPE, E_NULL, E_SEQ, E_SHAPE, E_VALUE, E_WS, HEADER

FORWARD = ["x", "dt", "A", "B", "C", "D", "z", "act", "init", "y", "final", "states"]
BACKWARD = ["dy", "dfinal", "x", "dt", "A", "B", "C", "D", "z", "act", "init", "states", "dx", "ddt", "dA", "dB", "dC",
            "dD", "dz", "ddt_bias", "dinit"]
STEP = ["state", "state_out", "x", "dt", "A", "B", "C", "D", "z", "act", "y"]


@pytest.fixture(scope="module")
def lib():
    return ops._lib()


def shape(**kw):
    s = sel._SelectiveShape()
    for k, v in {**dict(batch=2, seqlen=100, channels=64, dstate=16, ngroups=2, dtype=1, ydtype=1), **kw}.items():
        setattr(s, k, v)
    return s


def act(bias=True, lo=0.0, hi=float("inf"), where=None):
    return ctypes.byref(_DtAct((at(50) if where is None else where) if bias else None, lo, hi))


def runs(lib):
    """The three calls, each of a shape and what is to be other than usual."""
    def make(f, names, ws):
        def go(sh=None, **kw):
            kw.setdefault("act", act())
            return call(f, names, shape() if sh is None else sh, **{"ws": ws, **kw})
        return go
    return (make(lib.ssd_selective_scan, FORWARD, True), make(lib.ssd_selective_scan_backward, BACKWARD, True),
            make(lib.ssd_selective_scan_step, STEP, False))


def test_shapes(lib):
    fwd, bwd, step = runs(lib)
    for f, names, ws in ((lib.ssd_selective_scan, FORWARD, True), (lib.ssd_selective_scan_backward, BACKWARD, True),
                         (lib.ssd_selective_scan_step, STEP, False)):
        assert call(f, names, None, ws=ws, act=act()) == E_NULL
    for f in (fwd, bwd, step):
        assert f(shape(dtype=2)) == E_DTYPE and f(shape(ydtype=-1)) == E_DTYPE
        assert f(shape(reserved=1)) == E_SHAPE
        for c in (0, 4, 12, 2 ** 20 + 8, -8):
            assert f(shape(channels=c)) == E_SHAPE, c
        for n in (0, -1, 65):
            assert f(shape(dstate=n)) == E_SHAPE, n
        for g in (0, -2, 3, 128):
            assert f(shape(ngroups=g)) == E_SHAPE, g
        assert f(shape(channels=2 ** 20, ngroups=2 ** 20, dstate=8)) == E_SHAPE  # a row of B over 2^22
        for b in (-1, 2 ** 24 + 1):
            assert f(shape(batch=b)) == E_SHAPE
        for name in ("x_stride", "dt_stride", "z_stride", "dx_stride", "ddt_stride", "dz_stride"):
            for v in (-64, 8, 56, 68):
                assert f(shape(**{name: v})) == E_SHAPE, (name, v)
        for name in ("b_stride", "c_stride", "db_stride", "dc_stride"):
            for v in (-32, 1, 31):
                assert f(shape(**{name: v})) == E_SHAPE, (name, v)
        assert f(act=act(lo=-1.0)) == E_VALUE and f(act=act(lo=float("nan"))) == E_VALUE
        assert f(act=act(lo=2.0, hi=1.0)) == E_VALUE and f(act=act(hi=float("nan"))) == E_VALUE
        assert f(act=act(lo=float("inf"))) == E_VALUE
        for name in ("x", "dt", "A", "B", "C"):
            assert f(**{name: None}) == E_NULL, name
        for name in ("x", "dt", "z"):
            assert f(**{name: at(30) + 8}) == E_ALIGN, name
        for name in ("A", "D"):
            assert f(**{name: at(30) + 2}) == E_ALIGN, name
        for name in ("B", "C"):
            assert f(**{name: at(30) + 1}) == E_ALIGN, name
            assert f(shape(dtype=0), **{name: at(30) + 2}) == E_ALIGN, name
        assert f(act=act(where=at(50) + 2)) == E_ALIGN
    for f in (fwd, bwd):
        for name in ("x_stride", "dx_stride", "c_stride", "db_stride"):
            assert f(shape(**{name: 2 ** 22 + 8})) == E_SHAPE, name
        assert f(shape(seqlen=-1)) == E_SHAPE
        assert f(shape(batch=2 ** 20, seqlen=2 ** 12)) == E_SHAPE
        assert f(shape(batch=2 ** 24, seqlen=1, channels=2 ** 16, dstate=64, ngroups=1)) == E_SHAPE  # states over 2^40
        host = (ctypes.c_int32 * 3)(0, 60, 40)
        assert f(shape(cu_seqlens=at(41), cu_seqlens_host=ctypes.addressof(host))) == E_SEQ
        host[:] = [0, 60, 101]
        assert f(shape(cu_seqlens=at(41), cu_seqlens_host=ctypes.addressof(host))) == E_SEQ
        assert f(shape(cu_seqlens_host=ctypes.addressof(host))) == E_SHAPE
        assert f(shape(batch=0, cu_seqlens=at(41))) == E_SHAPE


def need(lib, sh, backward):
    n = ctypes.c_size_t(0)
    assert lib.ssd_selective_scan_workspace_size(ctypes.byref(sh), backward, ctypes.byref(n)) == 0
    return n.value


def test_workspace(lib):
    fwd, bwd, _ = runs(lib)
    long = shape(batch=1, seqlen=4096)  # one sequence over many items
    for f, backward in ((fwd, 0), (bwd, 1)):
        n = need(lib, long, backward)
        assert n > 0
        assert f(long, size=n - 1) == E_WS and f(long, ws=None) == E_WS and f(long, ws=at(40) + 8) == E_ALIGN
    assert lib.ssd_selective_scan_workspace_size(ctypes.byref(long), 2, ctypes.byref(ctypes.c_size_t())) == E_VALUE
    assert lib.ssd_selective_scan_workspace_size(ctypes.byref(long), 0, None) == E_NULL


def test_outputs(lib):
    fwd, bwd, step = runs(lib)
    for name in FORWARD:
        k = FORWARD.index(name)
        if name in ("x", "dt", "A", "B", "C", "D", "z", "init"):
            assert fwd(y=at(k)) == E_SHAPE and fwd(final=at(k)) == E_SHAPE and fwd(states=at(k)) == E_SHAPE, name
    assert fwd(y=None) == E_NULL and fwd(y=at(30) + 8) == E_ALIGN and fwd(final=at(9)) == E_SHAPE
    for name in ("dy", "states", "dx", "ddt", "dA", "dB", "dC", "dz"):
        assert bwd(**{name: None}) == E_NULL, name
    for name, other in (("dx", 2), ("ddt", 0), ("dB", 16), ("dC", 6), ("dD", 14), ("dz", 12), ("ddt_bias", 4),
                        ("dinit", 1), ("dA", 11)):
        assert bwd(**{name: at(other)}) == E_SHAPE, name
    assert bwd(z=None) == E_SHAPE  # dz without z
    assert bwd(D=None) == E_SHAPE and bwd(act=None) == E_SHAPE and bwd(act=act(bias=False)) == E_SHAPE
    for name in ("state", "state_out", "y"):
        assert step(**{name: None}) == E_NULL, name
    assert step(y=at(0)) == E_SHAPE and step(state_out=at(2)) == E_SHAPE and step(state_out=at(0), y=at(0)) == E_SHAPE
    assert step(shape(batch=0), state_out=at(0)) == 0


def test_binding():
    m = re.search(r"#define SSD_SELECTIVE_STATE_ROWS (\d+)", open(HEADER).read())
    assert m and int(m.group(1)) == sel.SELECTIVE_STATE_ROWS
    x, A, B = torch.zeros(1, 4, 8), torch.zeros(8, 16), torch.zeros(1, 4, 1, 16)
    with pytest.raises(ValueError):
        ssd.selective_scan(x, x, A, B, B)
    with pytest.raises(ValueError):
        ssd.selective_scan_backward(x, x, x, A, B, B, A)
    with pytest.raises(ValueError):
        ssd.selective_scan_step(A[None], x[:, 0], x[:, 0], A, B[:, 0], B[:, 0])
    for bad in (dict(dt_bias=torch.zeros(8)), dict(dt_limit=(0, 1))):
        with pytest.raises(ValueError):
            sel._activation(False, bad.get("dt_bias"), bad.get("dt_limit"), 8)


def test_shapes_of_the_binding():
    """What _shape refuses and how it reads strides (no device is touched)."""
    ops._lib()
    w = torch.zeros(2, 5, 80)
    x, A = torch.zeros(2, 5, 8), torch.zeros(8, 11)
    B, C = (t.unflatten(-1, (2, 11)) for t in w[..., 3:47].split(22, -1))
    sh = sel._shape(x, x, A, B, C, None, None, torch.float32)
    assert (sh.b_stride, sh.c_stride, sh.x_stride, sh.dstate, sh.ngroups) == (80, 80, 0, 11, 2)
    assert sel._state_stride(torch.zeros(3, 4, 1, 16), "B") == 0
    assert sel._state_stride(w[:, 1, :16].unflatten(-1, (1, 16)), "B") == 400
    for bad in (w[..., :32].unflatten(-1, (2, 16)).transpose(-1, -2), w[..., :64:2].unflatten(-1, (2, 16)),
                w[..., :32].unflatten(-1, (2, 16)).transpose(0, 1), w[:, :3, :16].unflatten(-1, (1, 16))):
        with pytest.raises(ValueError):
            sel._state_stride(bad, "B")
    for args in ((x, x[..., :4], A, B, C), (x, x, A, B[:, :4], C), (x, x, A, B, C[..., :5]), (x, x, A[:, :5], B, C),
                 (x, x, A, B[:, 0], C)):
        with pytest.raises(ValueError):
            sel._shape(*args, None, None, torch.float32)
    for args in ((x, x.bfloat16(), A, B, C), (x, x, A.double(), B, C), (x, x, A, B.bfloat16(), C)):
        with pytest.raises(TypeError):
            sel._shape(*args, None, None, torch.float32)
    with pytest.raises(SsdError):
        sel._scan_bytes(1, 1, 8, 65, 1, False, 0)
