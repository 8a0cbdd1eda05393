"""Host-side checks of the layer norm's entry points, and its oracle's gradients
against differences."""
import ctypes

import numpy as np
import pytest
import torch

import mamba_ssd_chunked_02_amd as ssd
from mamba_ssd_chunked_02_amd import block_ops as ops
from oracle import block
from test_abi_block import E_UNSUPPORTED, at, call, norm_shape
from test_abi_host import E_ALIGN, E_DTYPE, E_NULL, E_SHAPE, E_VALUE, E_WS
from test_block_oracle import differences

FORWARD = ["x", "residual", "weight", "bias", "scale", "y", "out", "mean", "rstd"]
BACKWARD = ["dy", "dout", "out", "weight", "mean", "rstd", "x", "scale", "dx", "dresidual", "dweight", "dbias", "dscale"]


@pytest.fixture(scope="module")
def lib():
    return ops._lib()


def test_refusals(lib):
    optional = {"scale", "bias", "dbias", "dscale", "dout", "dresidual"}
    for f, names, ws in ((lib.ssd_layer_norm, FORWARD, False), (lib.ssd_layer_norm_backward, BACKWARD, True)):
        go = lambda sh=None, **kw: call(f, names, norm_shape() if sh is None else sh, **{"ws": ws, **kw})  # noqa: E731
        assert call(f, names, None, ws=ws) == E_NULL
        assert go(norm_shape(dtype=3)) == E_DTYPE and go(norm_shape(dtype2=-1)) == E_DTYPE
        assert go(norm_shape(reserved=1)) == E_SHAPE and go(norm_shape(norm_before_gate=1)) == E_VALUE
        for eps in (-1e-6, float("nan"), float("inf")):
            assert go(norm_shape(eps=eps)) == E_VALUE
        for c in (0, -8, 4, 12):
            assert go(norm_shape(columns=c)) == E_SHAPE, c
        assert go(norm_shape(columns=16392)) == E_UNSUPPORTED
        assert go(norm_shape(rows=-1)) == E_SHAPE and go(norm_shape(rows=2 ** 31)) == E_SHAPE
        assert go(norm_shape(dtype=0, dtype2=1)) == E_UNSUPPORTED
        assert go(norm_shape(groups=2)) == E_SHAPE and go(norm_shape(x_stride=64)) == E_SHAPE
        for k, name in enumerate(names):
            if name not in optional | {"residual"} and not (name in ("mean", "rstd") and not ws):
                assert go(**{name: None}) == E_NULL, name
            assert go(**{name: at(30) + 4}) == E_ALIGN, name
        for name in ("y", "mean", "rstd") if not ws else ("dx", "dweight", "dbias", "dscale", "dresidual"):
            assert go(**{name: at(names.index("weight"))}) == E_SHAPE, name
    alone = dict(residual=None, scale=None, out=None)
    fwd = lambda sh=None, **kw: call(lib.ssd_layer_norm, FORWARD, norm_shape() if sh is None else sh, ws=False, **kw)  # noqa: E731
    assert fwd(**{**alone, "scale": at(4)}) == E_SHAPE and fwd(**{**alone, "out": at(6)}) == E_SHAPE
    assert fwd(norm_shape(dtype2=0), **alone) == E_DTYPE
    assert fwd(**{**alone, "y": at(0)}) == E_SHAPE
    # in place of the residual: out alone
    assert fwd(out=at(0)) == E_SHAPE and fwd(out=at(1), y=at(1)) == E_SHAPE and fwd(out=at(1), mean=at(1)) == E_SHAPE
    assert fwd(norm_shape(dtype2=0), out=at(1), x=at(1)) == E_SHAPE
    assert fwd(norm_shape(rows=0), out=at(1)) == 0 and fwd(norm_shape(rows=0), **alone) == 0
    bwd = lambda sh=None, **kw: call(lib.ssd_layer_norm_backward, BACKWARD, norm_shape() if sh is None else sh, **kw)  # noqa: E731
    assert bwd(scale=None) == E_SHAPE and bwd(size=8) == E_WS and bwd(ws=None) == E_WS
    assert bwd(dx=at(0)) == E_SHAPE and bwd(norm_shape(dtype2=0), dx=at(1)) == E_SHAPE
    for kw in (dict(dx=at(1)), dict(dresidual=at(1)), dict(dx=at(1), dy=at(1)), dict(dresidual=at(1), out=at(1))):
        assert bwd(size=8, **kw) == E_WS, kw
    assert bwd(dx=at(1), dresidual=at(1)) == E_SHAPE
    n = ctypes.c_size_t(0)
    assert lib.ssd_layer_norm_backward_workspace_size(ctypes.byref(norm_shape()), ctypes.byref(n)) == 0
    assert n.value >= 3 * 64 * 4
    assert lib.ssd_layer_norm_backward_workspace_size(ctypes.byref(norm_shape()), None) == E_NULL


def test_binding_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    for f in (lambda: ssd.layer_norm(x, w), lambda: ssd.add_layer_norm(x, x, w), lambda: ssd.add_layer_norm(x, None, w),
              lambda: ssd.layer_norm_backward(x, x, w, w, w), lambda: ssd.add_layer_norm_backward(x, x, w, w, w)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        ssd.layer_norm_backward(x, x.bfloat16(), w, w, w)


@pytest.mark.parametrize("residual,scaled", [(True, True), (True, False), (False, False)])
def test_oracle_gradients(residual, scaled):
    rng, rows, D = np.random.default_rng(2), 3, 8
    a = {"x": rng.standard_normal((rows, D)), "weight": rng.standard_normal(D), "bias": rng.standard_normal(D)}
    if residual:
        a["residual"] = rng.standard_normal((rows, D)) + 1
    if scaled:
        a["scale"] = rng.standard_normal(D)
    dy, dout = rng.standard_normal((rows, D)), rng.standard_normal((rows, D)) if residual else None

    def f():
        y, u, _, _ = block.layer_norm(a["x"], a["weight"], a["bias"], a.get("residual"), a.get("scale"))
        return (y * dy).sum() + (0 if dout is None else (u * dout).sum())
    _, u, mean, rstd = block.layer_norm(a["x"], a["weight"], a["bias"], a.get("residual"), a.get("scale"))
    g, s = block.layer_norm_backward(dy, u, a["weight"], mean, rstd, dout, a["x"], a.get("scale"))
    for name in a:
        differences(f, a, name, g["d" + name])
        assert (np.abs(g["d" + name]) <= s["d" + name] * (1 + 1e-12)).all(), name
