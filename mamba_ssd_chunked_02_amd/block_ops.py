"""The operators around the scan in a trained or served block: the gated
linear recurrence, the residual and gated RMS norms, and the gradients of the
causal conv1d (``include/ssd.h``).

    y, final = gated_scan(x, r, i, lam)                       # + gated_scan_step, gated_scan_backward
    y, residual = add_rms_norm(x, residual, weight, scale=s)  # + add_rms_norm_backward
    y = gated_rms_norm(x, z, weight)                          # + gated_rms_norm_backward
    dx, dweight, dbias, dstate = causal_conv1d_backward(dys, x, weight, bias)

Like the rest of the binding they marshal arguments only, run on torch's
current stream of the tensors' device, and record no autograd graph: a
training step calls the backward functions, which take the forward's inputs
and what it returned.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

from . import (_check, _conv_outputs, _ConvShape, _dtype_code, _dtype_code_of, _expect, _ptr, _stream_handle, _torch,
               load)

__all__ = ["gated_scan", "gated_scan_step", "gated_scan_backward", "add_rms_norm", "add_rms_norm_backward",
           "gated_rms_norm", "gated_rms_norm_backward", "causal_conv1d_backward", "GATED_TILE_ROWS"]

GATED_TILE_ROWS = 128  # SSD_GATED_TILE_ROWS of include/ssd.h


class _GatedShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("ydtype", ctypes.c_int32), ("rate", ctypes.c_float),
                ("x_stride", ctypes.c_int64), ("r_stride", ctypes.c_int64), ("i_stride", ctypes.c_int64),
                ("dx_stride", ctypes.c_int64), ("dr_stride", ctypes.c_int64), ("di_stride", ctypes.c_int64),
                ("reserved", ctypes.c_int64), ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_host", ctypes.c_void_p)]


class _NormShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("columns", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("dtype2", ctypes.c_int32), ("eps", ctypes.c_float),
                ("norm_before_gate", ctypes.c_int32), ("x_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64),
                ("dx_stride", ctypes.c_int64), ("dz_stride", ctypes.c_int64), ("reserved", ctypes.c_int64)]


_declared = False


def _lib():
    global _declared
    lib = load()
    if not _declared:
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        szp = ctypes.POINTER(sz)
        gsp, nsp, csp = (ctypes.POINTER(t) for t in (_GatedShape, _NormShape, _ConvShape))
        for name, args in {
                "ssd_gated_scan_workspace_size": [gsp, ctypes.c_int32, szp],
                "ssd_gated_scan": [vp] * 8 + [gsp, vp, sz, vp],
                "ssd_gated_scan_backward": [vp] * 13 + [gsp, vp, sz, vp],
                "ssd_gated_scan_step": [vp] * 7 + [gsp, vp],
                "ssd_norm_backward_workspace_size": [nsp, szp],
                "ssd_add_rms_norm": [vp] * 7 + [nsp, vp],
                "ssd_add_rms_norm_backward": [vp] * 11 + [nsp, vp, sz, vp],
                "ssd_gated_rms_norm": [vp] * 5 + [nsp, vp],
                "ssd_gated_rms_norm_backward": [vp] * 8 + [nsp, vp, sz, vp],
                "ssd_causal_conv1d_backward_workspace_size": [csp, szp],
                "ssd_causal_conv1d_backward": [vp] * 10 + [csp, vp, sz, vp]}.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = ctypes.c_int32
        _declared = True
    return lib


def _same_device(first, *others):
    """All tensors on one GPU; returns that device."""
    for t in (first,) + others:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on the GPU")
        if t.device != first.device:
            raise ValueError("tensors live on %s and %s" % (first.device, t.device))
    return first.device


def _row_stride(t, name) -> int:
    """Elements from one row [C] of t to the next; the rows of all leading
    dimensions must lie at one distance (a column range of a wider tensor does)."""
    if t.numel() == 0:
        return 0
    if t.shape[-1] != 1 and t.stride(-1) != 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)
    rows, stride = 1, 0
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if rows == 1:
            stride = s
        elif s != rows * stride:
            raise ValueError("the rows of %s are not evenly spaced" % name)
        rows *= n
    if rows > 1 and stride < t.shape[-1]:
        raise ValueError("the rows of %s overlap" % name)
    return stride if rows > 1 else 0


def _shaped(t, shape, dtype, name):
    """Shape and dtype; the strides are free."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))


def _out(t, shape, dtype, name, device):
    """A given output, checked, or a new one."""
    torch = _torch()
    if t is None:
        return torch.empty(tuple(shape), dtype=dtype, device=device)
    _shaped(t, shape, dtype, name)
    return t


def _workspace(given, need, device):
    torch = _torch()
    if given is None or given.numel() * given.element_size() < need:
        return torch.empty(int(need), dtype=torch.uint8, device=device)
    return given


def _bytes(w) -> int:
    return w.numel() * w.element_size()


def _sequences(sh, x, cu_seqlens, cu_seqlens_host):
    """Fills batch, seqlen and the offsets of a shape from x [b, L, C] or [T, C]; returns what must stay alive."""
    torch = _torch()
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError("dense tensors must be [b, L, C]")
        if cu_seqlens_host is not None:
            raise ValueError("cu_seqlens_host without cu_seqlens")
        sh.batch, sh.seqlen = x.shape[0], x.shape[1]
        return None
    if x.dim() != 2:
        raise ValueError("packed tensors must be [T, C]")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [nseq + 1]")
    _expect(cu_seqlens, (cu_seqlens.shape[0],), torch.int32, "cu_seqlens")
    sh.batch, sh.seqlen = cu_seqlens.shape[0] - 1, x.shape[0]
    sh.cu_seqlens = cu_seqlens.data_ptr()
    if cu_seqlens_host is None:
        return None
    import numpy as np
    keep = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int32))
    if keep.shape != (sh.batch + 1,):
        raise ValueError("cu_seqlens_host has shape %s, expected %s" % (keep.shape, (sh.batch + 1,)))
    sh.cu_seqlens_host = keep.ctypes.data
    return keep


# ------------------------------------------------------------------ gated recurrence
def _gated_shape(x, r, i, lam, rate, y_dtype):
    torch = _torch()
    sh = _GatedShape()
    C = x.shape[-1]
    sh.channels = C
    sh.dtype, sh.ydtype = _dtype_code(x), _dtype_code_of(y_dtype)
    sh.rate = float(rate)
    for name, t in (("x", x), ("r", r), ("i", i)):
        _shaped(t, x.shape, x.dtype, name)
        setattr(sh, name + "_stride", _row_stride(t, name))
    _expect(lam, (C,), torch.float32, "lam")
    return sh


def gated_scan(x, r, i, lam, *, rate: float = 8.0, init_state=None, cu_seqlens=None,
               cu_seqlens_host: Optional[Sequence[int]] = None, y=None, final_state=None, want_final: bool = True,
               want_states: bool = False, workspace=None, y_dtype=None):
    """Gated linear recurrence over whole sequences, per channel:

        log a = -rate softplus(lam) sigmoid(r),  h = a h + sqrt(1 - a^2) sigmoid(i) x,  y = h

    x, r, i: dense [b, L, C] or packed [T, C] with ``cu_seqlens`` (int32 GPU
    tensor [b + 1]), fp32 or bf16; each may be a column range of a wider
    tensor.  lam [C] fp32; ``init_state`` [b, C] fp32 or None (zero).
    Returns (y, final_state), y of x's dtype unless ``y_dtype`` says fp32 or
    bf16, final_state [b, C] fp32 (None with ``want_final=False``); with
    ``want_states`` (y, final_state, states), the fp32 states that
    gated_scan_backward needs, [ceil(rows / GATED_TILE_ROWS), C].

    A sequence of no tokens passes its state through.  Rows behind the last
    sequence of a packed batch are left as they were in y."""
    torch = _torch()
    dev = _same_device(x, r, i, lam, init_state, cu_seqlens, y, final_state, workspace)
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    sh = _gated_shape(x, r, i, lam, rate, y_dtype)
    keep = _sequences(sh, x, cu_seqlens, cu_seqlens_host)
    n, C, rows = sh.batch, sh.channels, math.prod(x.shape[:-1])
    _expect(init_state, (n, C), torch.float32, "init_state")
    _expect(y, x.shape, y_dtype, "y")
    _expect(final_state, (n, C), torch.float32, "final_state")
    lib = _lib()
    with torch.cuda.device(dev):
        y = _out(y, x.shape, y_dtype, "y", dev)
        if final_state is None and want_final:
            final_state = torch.empty((n, C), dtype=torch.float32, device=dev)
        states = None
        if want_states:
            states = torch.empty((-(-rows // GATED_TILE_ROWS), C), dtype=torch.float32, device=dev)
        need = ctypes.c_size_t(0)
        _check(lib.ssd_gated_scan_workspace_size(ctypes.byref(sh), 0, ctypes.byref(need)), "ssd_gated_scan_workspace_size")
        workspace = _workspace(workspace, need.value, dev)
        _check(lib.ssd_gated_scan(x.data_ptr(), r.data_ptr(), i.data_ptr(), _ptr(lam), _ptr(init_state), _ptr(y),
                                  _ptr(final_state), _ptr(states), ctypes.byref(sh), _ptr(workspace),
                                  _bytes(workspace), _stream_handle(x)), "ssd_gated_scan")
    del keep
    return (y, final_state, states) if want_states else (y, final_state)


def gated_scan_backward(dy, x, r, i, lam, states, *, rate: float = 8.0, init_state=None, dfinal_state=None,
                        cu_seqlens=None, cu_seqlens_host: Optional[Sequence[int]] = None, dx=None, dr=None, di=None,
                        dlam=None, dinit_state=None, want_dinit: bool = True, workspace=None):
    """Gradients of gated_scan for dy (fp32 or bf16, shaped as x) and
    ``dfinal_state`` [b, C] fp32 (None: zero).  x, r, i, lam, ``rate``,
    ``init_state`` and the offsets as given to gated_scan, ``states`` as
    returned by it.  Returns (dx, dr, di, dlam, dinit_state); dx, dr and di may
    be given as column ranges of one wider tensor.  Rows behind the last
    sequence of a packed batch are left as they were in dx, dr and di."""
    torch = _torch()
    dev = _same_device(x, dy, r, i, lam, states, init_state, dfinal_state, cu_seqlens, dx, dr, di, dlam, dinit_state,
                       workspace)
    sh = _gated_shape(x, r, i, lam, rate, dy.dtype)
    keep = _sequences(sh, x, cu_seqlens, cu_seqlens_host)
    n, C, rows = sh.batch, sh.channels, math.prod(x.shape[:-1])
    _expect(dy, x.shape, dy.dtype, "dy")
    _expect(states, (-(-rows // GATED_TILE_ROWS), C), torch.float32, "states")
    _expect(init_state, (n, C), torch.float32, "init_state")
    _expect(dfinal_state, (n, C), torch.float32, "dfinal_state")
    _expect(dlam, (C,), torch.float32, "dlam")
    _expect(dinit_state, (n, C), torch.float32, "dinit_state")
    lib = _lib()
    with torch.cuda.device(dev):
        grads = []
        for name, t in (("dx", dx), ("dr", dr), ("di", di)):
            t = _out(t, x.shape, x.dtype, name, dev)
            setattr(sh, name + "_stride", _row_stride(t, name))
            grads.append(t)
        dlam = _out(dlam, (C,), torch.float32, "dlam", dev)
        if dinit_state is None and want_dinit:
            dinit_state = torch.empty((n, C), dtype=torch.float32, device=dev)
        need = ctypes.c_size_t(0)
        _check(lib.ssd_gated_scan_workspace_size(ctypes.byref(sh), 1, ctypes.byref(need)), "ssd_gated_scan_workspace_size")
        workspace = _workspace(workspace, need.value, dev)
        _check(lib.ssd_gated_scan_backward(_ptr(dy), _ptr(dfinal_state), x.data_ptr(), r.data_ptr(), i.data_ptr(),
                                           _ptr(lam), _ptr(init_state), _ptr(states), *[t.data_ptr() for t in grads],
                                           _ptr(dlam), _ptr(dinit_state), ctypes.byref(sh), _ptr(workspace),
                                           _bytes(workspace), _stream_handle(x)), "ssd_gated_scan_backward")
    del keep
    return (*grads, dlam, dinit_state)


def gated_scan_step(state, x, r, i, lam, *, rate: float = 8.0, state_out=None, y=None, y_dtype=None):
    """One token per sequence: x, r, i [b, C]; ``state`` [b, C] fp32 is updated
    in place, or left as it is and the new one written to ``state_out``.
    Returns y [b, C], of x's dtype unless ``y_dtype`` says otherwise."""
    torch = _torch()
    dev = _same_device(x, r, i, lam, state, state_out, y)
    if x.dim() != 2:
        raise ValueError("one token per sequence: x must be [b, C]")
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    sh = _gated_shape(x, r, i, lam, rate, y_dtype)
    sh.batch, sh.seqlen = x.shape[0], 1
    _expect(state, x.shape, torch.float32, "state")
    _expect(state_out, x.shape, torch.float32, "state_out")
    _expect(y, x.shape, y_dtype, "y")
    with torch.cuda.device(dev):
        y = _out(y, x.shape, y_dtype, "y", dev)
        _check(_lib().ssd_gated_scan_step(_ptr(state), _ptr(state if state_out is None else state_out), x.data_ptr(),
                                          r.data_ptr(), i.data_ptr(), _ptr(lam), _ptr(y), ctypes.byref(sh),
                                          _stream_handle(x)), "ssd_gated_scan_step")
    return y


# ------------------------------------------------------------------ norms
def _norm_shape(rows, D, dtype, dtype2, eps, groups=1, norm_before_gate=False):
    sh = _NormShape()
    sh.rows, sh.columns, sh.groups = rows, D, int(groups)
    sh.dtype, sh.dtype2 = _dtype_code_of(dtype), _dtype_code_of(dtype2)
    sh.eps = float(eps)
    sh.norm_before_gate = 1 if norm_before_gate else 0
    return sh


def _norm_workspace(sh, workspace, device):
    need = ctypes.c_size_t(0)
    _check(_lib().ssd_norm_backward_workspace_size(ctypes.byref(sh), ctypes.byref(need)),
           "ssd_norm_backward_workspace_size")
    return _workspace(workspace, need.value, device)


def add_rms_norm(x, residual, weight, *, scale=None, eps: float = 1e-5, y=None, residual_out=None,
                 want_rstd: bool = False):
    """Residual addition and the RMS norm in front of the next block:

        residual_out = residual + scale * x,  y = residual_out / rms(residual_out) * weight

    x [..., D] fp32 or bf16, residual of x's shape in x's dtype or fp32,
    weight [D] fp32, ``scale`` [D] fp32 or None (1).  ``residual_out`` may be
    residual itself.  The norm is that of the fp32 sum, before residual_out is
    rounded.  Returns (y, residual_out), or (y, residual_out, rstd [...] fp32)
    with ``want_rstd``, which add_rms_norm_backward needs."""
    torch = _torch()
    dev = _same_device(x, residual, weight, scale, y, residual_out)
    D, lead = x.shape[-1], x.shape[:-1]
    _expect(x, x.shape, x.dtype, "x")
    _expect(residual, x.shape, residual.dtype, "residual")
    _expect(weight, (D,), torch.float32, "weight")
    _expect(scale, (D,), torch.float32, "scale")
    _expect(y, x.shape, x.dtype, "y")
    _expect(residual_out, x.shape, residual.dtype, "residual_out")
    sh = _norm_shape(math.prod(lead), D, x.dtype, residual.dtype, eps)
    with torch.cuda.device(dev):
        y = _out(y, x.shape, x.dtype, "y", dev)
        residual_out = _out(residual_out, x.shape, residual.dtype, "residual_out", dev)
        rstd = torch.empty(tuple(lead), dtype=torch.float32, device=dev) if want_rstd else None
        _check(_lib().ssd_add_rms_norm(_ptr(x), _ptr(residual), _ptr(weight), _ptr(scale), _ptr(y), _ptr(residual_out),
                                       _ptr(rstd), ctypes.byref(sh), _stream_handle(x)), "ssd_add_rms_norm")
    return (y, residual_out, rstd) if want_rstd else (y, residual_out)


def add_rms_norm_backward(dy, residual_out, weight, rstd, *, dresidual_out=None, x=None, scale=None, dx=None,
                          dresidual=None, workspace=None):
    """Gradients of add_rms_norm for dy (x's dtype) and ``dresidual_out``
    (residual's dtype; None: zero), from its residual_out and rstd.  With
    ``scale``, x is needed for its gradient.  Returns (dx, dresidual, dweight,
    dscale or None); without a scale and with one dtype dx and dresidual are
    the same tensor unless both are given."""
    torch = _torch()
    dev = _same_device(dy, residual_out, weight, rstd, dresidual_out, x, scale, dx, dresidual, workspace)
    D = dy.shape[-1]
    if scale is not None and x is None:
        raise ValueError("the gradient of scale needs x")
    rdt = residual_out.dtype
    _expect(dy, dy.shape, dy.dtype, "dy")
    _expect(residual_out, dy.shape, rdt, "residual_out")
    _expect(weight, (D,), torch.float32, "weight")
    _expect(rstd, dy.shape[:-1], torch.float32, "rstd")
    _expect(dresidual_out, dy.shape, rdt, "dresidual_out")
    _expect(x, dy.shape, dy.dtype, "x")
    _expect(scale, (D,), torch.float32, "scale")
    _expect(dx, dy.shape, dy.dtype, "dx")
    _expect(dresidual, dy.shape, rdt, "dresidual")
    sh = _norm_shape(math.prod(dy.shape[:-1]), D, dy.dtype, rdt, 0.0)
    with torch.cuda.device(dev):
        one = scale is None and rdt == dy.dtype and (dx is None or dresidual is None)
        if one:
            dx = dresidual = _out(dx if dresidual is None else dresidual, dy.shape, rdt, "dx", dev)
        else:
            dx = _out(dx, dy.shape, dy.dtype, "dx", dev)
            dresidual = _out(dresidual, dy.shape, rdt, "dresidual", dev)
        dweight = torch.empty(D, dtype=torch.float32, device=dev)
        dscale = None if scale is None else torch.empty(D, dtype=torch.float32, device=dev)
        workspace = _norm_workspace(sh, workspace, dev)
        _check(_lib().ssd_add_rms_norm_backward(
            _ptr(dy), _ptr(dresidual_out), _ptr(residual_out), _ptr(weight), _ptr(rstd),
            None if scale is None else _ptr(x), _ptr(scale), _ptr(dx), None if one else _ptr(dresidual), _ptr(dweight),
            _ptr(dscale), ctypes.byref(sh), _ptr(workspace), _bytes(workspace), _stream_handle(dy)),
            "ssd_add_rms_norm_backward")
    return dx, dresidual, dweight, dscale


def _gated_norm_inputs(x, z, weight, groups, eps, norm_before_gate):
    torch = _torch()
    D = x.shape[-1]
    _shaped(x, z.shape, x.dtype, "x")
    _expect(weight, (D,), torch.float32, "weight")
    sh = _norm_shape(math.prod(x.shape[:-1]), D, z.dtype, x.dtype, eps, groups, norm_before_gate)
    sh.x_stride, sh.z_stride = _row_stride(x, "x"), _row_stride(z, "z")
    return sh


def gated_rms_norm(x, z, weight, *, groups: int = 1, eps: float = 1e-5, norm_before_gate: bool = False, y=None,
                   want_rstd: bool = False):
    """RMS norm behind the scan with its gate: y = norm(x silu(z)) weight, or
    norm(x) weight silu(z) with ``norm_before_gate``; each of ``groups`` equal
    column ranges has its own mean.

    x [..., D] in z's dtype or fp32, z [..., D] fp32 or bf16 (each may be a
    column range of a wider tensor), weight [D] fp32.  Returns y (z's dtype),
    or (y, rstd [..., groups] fp32) with ``want_rstd``."""
    torch = _torch()
    dev = _same_device(x, z, weight, y)
    sh = _gated_norm_inputs(x, z, weight, groups, eps, norm_before_gate)
    _expect(y, x.shape, z.dtype, "y")
    with torch.cuda.device(dev):
        y = _out(y, x.shape, z.dtype, "y", dev)
        rstd = torch.empty(tuple(x.shape[:-1]) + (sh.groups,), dtype=torch.float32, device=dev) if want_rstd else None
        _check(_lib().ssd_gated_rms_norm(x.data_ptr(), z.data_ptr(), _ptr(weight), _ptr(y), _ptr(rstd),
                                         ctypes.byref(sh), _stream_handle(x)), "ssd_gated_rms_norm")
    return (y, rstd) if want_rstd else y


def gated_rms_norm_backward(dy, x, z, weight, rstd, *, groups: int = 1, norm_before_gate: bool = False, dx=None,
                            dz=None, workspace=None):
    """Gradients of gated_rms_norm for dy (z's dtype) from its inputs and rstd:
    (dx, dz, dweight).  dx and dz may be given as column ranges of a wider
    tensor."""
    torch = _torch()
    dev = _same_device(x, z, dy, weight, rstd, dx, dz, workspace)
    sh = _gated_norm_inputs(x, z, weight, groups, 0.0, norm_before_gate)
    _expect(dy, x.shape, z.dtype, "dy")
    _expect(rstd, tuple(x.shape[:-1]) + (sh.groups,), torch.float32, "rstd")
    with torch.cuda.device(dev):
        dx = _out(dx, x.shape, x.dtype, "dx", dev)
        dz = _out(dz, x.shape, z.dtype, "dz", dev)
        sh.dx_stride, sh.dz_stride = _row_stride(dx, "dx"), _row_stride(dz, "dz")
        dweight = torch.empty(x.shape[-1], dtype=torch.float32, device=dev)
        workspace = _norm_workspace(sh, workspace, dev)
        _check(_lib().ssd_gated_rms_norm_backward(_ptr(dy), x.data_ptr(), z.data_ptr(), _ptr(weight), _ptr(rstd),
                                                  dx.data_ptr(), dz.data_ptr(), _ptr(dweight), ctypes.byref(sh),
                                                  _ptr(workspace), _bytes(workspace), _stream_handle(x)),
               "ssd_gated_rms_norm_backward")
    return dx, dz, dweight


# ------------------------------------------------------------------ conv1d gradients
def causal_conv1d_backward(dys, x, weight, bias=None, *, cu_seqlens=None, cu_seqlens_host=None, conv_state=None,
                           dfinal_conv_state=None, activation: bool = True, dx=None, want_dstate: Optional[bool] = None,
                           workspace=None):
    """Gradients of causal_conv1d for the gradients ``dys`` of its output parts
    (a list, in order; one dtype) and ``dfinal_conv_state`` [b, K-1, C] (x's
    dtype; None: zero).  The other arguments as given to causal_conv1d.

    Returns (dx, dweight [C, K] fp32, dbias [C] fp32 or None without a bias,
    dconv_state [b, K-1, C] or None); dconv_state is returned where conv_state
    is given, or as ``want_dstate`` says."""
    torch = _torch()
    dys = list(dys)
    if not dys:
        raise ValueError("no output parts")
    dev = _same_device(x, weight, bias, cu_seqlens, conv_state, dfinal_conv_state, dx, workspace, *dys)
    C, K = x.shape[-1], weight.shape[-1]
    _expect(x, x.shape, x.dtype, "x")
    _expect(weight, (C, K), torch.float32, "weight")
    _expect(bias, (C,), torch.float32, "bias")
    sh = _ConvShape()
    keep = _sequences(sh, x, cu_seqlens, cu_seqlens_host)
    n = sh.batch
    _expect(conv_state, (n, K - 1, C), x.dtype, "conv_state")
    _expect(dfinal_conv_state, (n, K - 1, C), x.dtype, "dfinal_conv_state")
    _expect(dx, x.shape, x.dtype, "dx")
    sh.channels, sh.width = C, K
    sh.dtype, sh.ydtype = _dtype_code(x), _dtype_code_of(dys[0].dtype)
    sh.activation = 1 if activation else 0
    if len(dys) > 3:
        raise ValueError("%d output parts, at most 3" % len(dys))
    co, _ = _conv_outputs(x.shape[:-1], C, [t.shape[-1] for t in dys], dys, dys[0].dtype, dev)
    lib = _lib()
    with torch.cuda.device(dev):
        dx = _out(dx, x.shape, x.dtype, "dx", dev)
        dweight = torch.empty((C, K), dtype=torch.float32, device=dev)
        dbias = None if bias is None else torch.empty(C, dtype=torch.float32, device=dev)
        want = conv_state is not None if want_dstate is None else want_dstate
        dstate = torch.empty((n, K - 1, C), dtype=x.dtype, device=dev) if want else None
        need = ctypes.c_size_t(0)
        _check(lib.ssd_causal_conv1d_backward_workspace_size(ctypes.byref(sh), ctypes.byref(need)),
               "ssd_causal_conv1d_backward_workspace_size")
        workspace = _workspace(workspace, need.value, dev)
        _check(lib.ssd_causal_conv1d_backward(ctypes.byref(co), _ptr(x), _ptr(weight), _ptr(bias), _ptr(conv_state),
                                              _ptr(dfinal_conv_state), _ptr(dx), _ptr(dweight), _ptr(dbias),
                                              _ptr(dstate), ctypes.byref(sh), _ptr(workspace), _bytes(workspace),
                                              _stream_handle(x)), "ssd_causal_conv1d_backward")
    del keep
    return dx, dweight, dbias, dstate
