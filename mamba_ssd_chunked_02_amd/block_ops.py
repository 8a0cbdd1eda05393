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
import functools
import math
from typing import Optional, Sequence

from . import (SSD_BF16, SSD_F32, SsdError, _conv_outputs, _ConvShape, _dtype_code_of, _expect, _torch, load)

__all__ = ["gated_scan", "gated_scan_step", "gated_scan_backward", "add_rms_norm", "add_rms_norm_backward",
           "gated_rms_norm", "gated_rms_norm_backward", "causal_conv1d_backward", "GATED_STATE_ROWS"]

GATED_STATE_ROWS = 64  # SSD_GATED_STATE_ROWS of include/ssd.h


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


_functions = {}
_codes = {}  # torch dtype -> ssd_dtype


def _lib():
    """The library, with the entry points below declared."""
    lib = load()
    if not _functions:
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        szp = ctypes.POINTER(sz)
        gsp, nsp, csp = (ctypes.POINTER(t) for t in (_GatedShape, _NormShape, _ConvShape))
        declared = {}
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
            declared[name] = f
        torch = _torch()
        _codes.update({torch.float32: SSD_F32, torch.bfloat16: SSD_BF16})
        _functions.update(declared)  # all at once: another thread sees none or every one
    return lib


def _fail(status, name):
    raise SsdError(status, name, load().ssd_last_error_detail().decode())


def _launch(index, name, *args):
    """Calls an entry point on the device's current stream, with the device current."""
    torch = _torch()
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch.cuda.current_device() == index:
        st = _functions[name](*args, stream)
    else:
        with torch.cuda.device(index):
            st = _functions[name](*args, stream)
    if st:
        _fail(st, name)


def _query(name, *args) -> int:
    need = ctypes.c_size_t(0)
    st = _functions[name](*args, ctypes.byref(need))
    if st:
        _fail(st, name)
    return need.value


# Workspace bytes: a function of the sizes alone, asked for once for each.
@functools.lru_cache(maxsize=1024)
def _gated_bytes(batch, seqlen, channels, packed, backward) -> int:
    sh = _GatedShape(batch, seqlen, channels, SSD_F32, SSD_F32, 1.0)
    sh.cu_seqlens = 16 if packed else None  # only whether there are offsets counts
    return _query("ssd_gated_scan_workspace_size", ctypes.byref(sh), backward)


@functools.lru_cache(maxsize=1024)
def _norm_bytes(rows, columns, groups) -> int:
    return _query("ssd_norm_backward_workspace_size", ctypes.byref(_NormShape(rows, columns, groups)))


@functools.lru_cache(maxsize=1024)
def _conv_bytes(batch, seqlen, channels, width, packed) -> int:
    sh = _ConvShape(batch, seqlen, channels, width)
    sh.cu_seqlens = 16 if packed else None
    return _query("ssd_causal_conv1d_backward_workspace_size", ctypes.byref(sh))


def _gpu(first, *others) -> int:
    """All tensors on one GPU; returns its index."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must live on the GPU")
    for t in others:
        if t is not None and t.get_device() != index:
            if not t.is_cuda:
                raise ValueError("tensors must live on the GPU")
            raise ValueError("tensors live on %s and %s" % (first.device, t.device))
    if not _functions:
        _lib()
    return index


def _code(dtype) -> int:
    code = _codes.get(dtype)
    return _dtype_code_of(dtype) if code is None else code


def _row_stride(t, name) -> int:
    """Elements from one row [C] of t to the next, 0 where the rows are dense; the
    rows of all leading dimensions must lie at one distance (a column range of
    a wider tensor does)."""
    if t.is_contiguous():
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
    if t.shape != shape or t.dtype != dtype:
        if tuple(t.shape) != tuple(shape):
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))


def _need(t, shape, dtype, name):
    """Shape, dtype and dense strides of a tensor that may be None."""
    if t is not None and (t.shape != shape or t.dtype != dtype or not t.is_contiguous()):
        _expect(t, shape, dtype, name)


def _p(t):
    return None if t is None else t.data_ptr()


def _new(like, shape, dtype):
    """A new dense tensor on `like`'s device."""
    if like.dtype == dtype and like.shape == shape and like.is_contiguous():
        return _torch().empty_like(like)
    return like.new_empty(shape, dtype=dtype)


def _workspace(given, need, like):
    if given is None or given.numel() * given.element_size() < need:
        return _new(like, (need,), _torch().uint8)
    if not given.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return given


def _bytes(w) -> int:
    return w.numel() * w.element_size()


def _sequences(sh, x, cu_seqlens, cu_seqlens_host):
    """Fills batch, seqlen and the offsets of a shape from x [b, L, C] or [T, C]; returns what must stay alive."""
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
    _need(cu_seqlens, cu_seqlens.shape, _torch().int32, "cu_seqlens")
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
    C, dtype = x.shape[-1], x.dtype
    _shaped(r, x.shape, dtype, "r")
    _shaped(i, x.shape, dtype, "i")
    _need(lam, (C,), _torch().float32, "lam")
    return _GatedShape(0, 0, C, _code(dtype), _code(y_dtype), rate, _row_stride(x, "x"), _row_stride(r, "r"),
                       _row_stride(i, "i"))


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
    gated_scan_backward needs, [ceil(rows / GATED_STATE_ROWS), C].

    A sequence of no tokens passes its state through.  Rows behind the last
    sequence of a packed batch are left as they were in y."""
    index = _gpu(x, r, i, lam, init_state, cu_seqlens, y, final_state, workspace)
    f32 = _torch().float32
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    sh = _gated_shape(x, r, i, lam, rate, y_dtype)
    keep = _sequences(sh, x, cu_seqlens, cu_seqlens_host)
    state = (sh.batch, sh.channels)
    _need(init_state, state, f32, "init_state")
    _need(y, x.shape, y_dtype, "y")
    _need(final_state, state, f32, "final_state")
    if y is None:
        y = _new(x, x.shape, y_dtype)
    if final_state is None and want_final:
        final_state = _new(x, state, f32)
    states = _new(x, _states_shape(x), f32) if want_states else None
    ref = ctypes.byref(sh)
    workspace = _workspace(workspace, _gated_bytes(sh.batch, sh.seqlen, sh.channels, cu_seqlens is not None, 0), x)
    _launch(index, "ssd_gated_scan", x.data_ptr(), r.data_ptr(), i.data_ptr(), lam.data_ptr(), _p(init_state),
            y.data_ptr(), _p(final_state), _p(states), ref, workspace.data_ptr(), _bytes(workspace))
    del keep
    return (y, final_state, states) if want_states else (y, final_state)


def _states_shape(x):
    return -(-math.prod(x.shape[:-1]) // GATED_STATE_ROWS), x.shape[-1]


def gated_scan_backward(dy, x, r, i, lam, states, *, rate: float = 8.0, init_state=None, dfinal_state=None,
                        cu_seqlens=None, cu_seqlens_host: Optional[Sequence[int]] = None, dx=None, dr=None, di=None,
                        dlam=None, dinit_state=None, want_dinit: bool = True, workspace=None):
    """Gradients of gated_scan for dy (fp32 or bf16, shaped as x) and
    ``dfinal_state`` [b, C] fp32 (None: zero).  x, r, i, lam, ``rate``,
    ``init_state`` and the offsets as given to gated_scan, ``states`` as
    returned by it.  Returns (dx, dr, di, dlam, dinit_state); dx, dr and di may
    be given as column ranges of one wider tensor.  Rows behind the last
    sequence of a packed batch are left as they were in dx, dr and di."""
    index = _gpu(x, dy, r, i, lam, states, init_state, dfinal_state, cu_seqlens, dx, dr, di, dlam, dinit_state,
                 workspace)
    f32 = _torch().float32
    sh = _gated_shape(x, r, i, lam, rate, dy.dtype)
    keep = _sequences(sh, x, cu_seqlens, cu_seqlens_host)
    state = (sh.batch, sh.channels)
    _need(dy, x.shape, dy.dtype, "dy")
    _need(states, _states_shape(x), f32, "states")
    _need(init_state, state, f32, "init_state")
    _need(dfinal_state, state, f32, "dfinal_state")
    _need(dlam, lam.shape, f32, "dlam")
    _need(dinit_state, state, f32, "dinit_state")
    grads = []
    for name, t in (("dx", dx), ("dr", dr), ("di", di)):
        if t is None:
            t = _new(x, x.shape, x.dtype)
        else:
            _shaped(t, x.shape, x.dtype, name)
            setattr(sh, name + "_stride", _row_stride(t, name))
        grads.append(t)
    if dlam is None:
        dlam = _new(lam, lam.shape, f32)
    if dinit_state is None and want_dinit:
        dinit_state = _new(x, state, f32)
    ref = ctypes.byref(sh)
    workspace = _workspace(workspace, _gated_bytes(sh.batch, sh.seqlen, sh.channels, cu_seqlens is not None, 1), x)
    _launch(index, "ssd_gated_scan_backward", dy.data_ptr(), _p(dfinal_state), x.data_ptr(), r.data_ptr(),
            i.data_ptr(), lam.data_ptr(), _p(init_state), states.data_ptr(), *[t.data_ptr() for t in grads],
            dlam.data_ptr(), _p(dinit_state), ref, workspace.data_ptr(), _bytes(workspace))
    del keep
    return (*grads, dlam, dinit_state)


def gated_scan_step(state, x, r, i, lam, *, rate: float = 8.0, state_out=None, y=None, y_dtype=None):
    """One token per sequence: x, r, i [b, C], dense or evenly spaced rows (the
    token's slice x[:, t] of a batch); ``state`` [b, C] fp32 is updated in place,
    or left as it is and the new one written to ``state_out``.
    Returns y [b, C], of x's dtype unless ``y_dtype`` says otherwise."""
    index = _gpu(x, r, i, lam, state, state_out, y)
    f32 = _torch().float32
    if x.dim() != 2:
        raise ValueError("one token per sequence: x must be [b, C]")
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    sh = _gated_shape(x, r, i, lam, rate, y_dtype)
    sh.batch = x.shape[0]
    _expect(state, x.shape, f32, "state")
    _need(state_out, x.shape, f32, "state_out")
    _need(y, x.shape, y_dtype, "y")
    if y is None:
        y = _new(x, x.shape, y_dtype)
    _launch(index, "ssd_gated_scan_step", state.data_ptr(), (state if state_out is None else state_out).data_ptr(),
            x.data_ptr(), r.data_ptr(), i.data_ptr(), lam.data_ptr(), y.data_ptr(), ctypes.byref(sh))
    return y


# ------------------------------------------------------------------ norms
def _norm_shape(t, dtype, dtype2, eps, groups=1, norm_before_gate=False, x_stride=0, z_stride=0):
    D = t.shape[-1]
    return _NormShape(t.numel() // D if D else 0, D, groups, _code(dtype), _code(dtype2), eps,
                      1 if norm_before_gate else 0, x_stride, z_stride)


def add_rms_norm(x, residual, weight, *, scale=None, eps: float = 1e-5, y=None, residual_out=None,
                 want_rstd: bool = False):
    """Residual addition and the RMS norm in front of the next block:

        residual_out = residual + scale * x,  y = residual_out / rms(residual_out) * weight

    x [..., D] fp32 or bf16, residual of x's shape in x's dtype or fp32,
    weight [D] fp32, ``scale`` [D] fp32 or None (1).  ``residual_out`` may be
    residual itself.  The norm is that of the fp32 sum, before residual_out is
    rounded.  Returns (y, residual_out), or (y, residual_out, rstd [...] fp32)
    with ``want_rstd``, which add_rms_norm_backward needs."""
    index = _gpu(x, residual, weight, scale, y, residual_out)
    f32, shape, dtype, rdtype = _torch().float32, x.shape, x.dtype, residual.dtype
    _need(x, shape, dtype, "x")
    _need(residual, shape, rdtype, "residual")
    _need(weight, shape[-1:], f32, "weight")
    _need(scale, shape[-1:], f32, "scale")
    _need(y, shape, dtype, "y")
    _need(residual_out, shape, rdtype, "residual_out")
    sh = _norm_shape(x, dtype, rdtype, eps)
    if y is None:
        y = _new(x, shape, dtype)
    if residual_out is None:
        residual_out = _new(x, shape, rdtype)
    rstd = _new(x, shape[:-1], f32) if want_rstd else None
    _launch(index, "ssd_add_rms_norm", x.data_ptr(), residual.data_ptr(), weight.data_ptr(), _p(scale), y.data_ptr(),
            residual_out.data_ptr(), _p(rstd), ctypes.byref(sh))
    return (y, residual_out, rstd) if want_rstd else (y, residual_out)


def add_rms_norm_backward(dy, residual_out, weight, rstd, *, dresidual_out=None, x=None, scale=None, dx=None,
                          dresidual=None, workspace=None):
    """Gradients of add_rms_norm for dy (x's dtype) and ``dresidual_out``
    (residual's dtype; None: zero), from its residual_out and rstd.  With
    ``scale``, x is needed for its gradient.  Returns (dx, dresidual, dweight,
    dscale or None); without a scale and with one dtype dx and dresidual are
    the same tensor unless both are given."""
    index = _gpu(dy, residual_out, weight, rstd, dresidual_out, x, scale, dx, dresidual, workspace)
    f32, shape, dtype, rdtype = _torch().float32, dy.shape, dy.dtype, residual_out.dtype
    if scale is not None and x is None:
        raise ValueError("the gradient of scale needs x")
    _need(dy, shape, dtype, "dy")
    _need(residual_out, shape, rdtype, "residual_out")
    _need(weight, shape[-1:], f32, "weight")
    _need(rstd, shape[:-1], f32, "rstd")
    _need(dresidual_out, shape, rdtype, "dresidual_out")
    _need(x, shape, dtype, "x")
    _need(scale, shape[-1:], f32, "scale")
    _need(dx, shape, dtype, "dx")
    _need(dresidual, shape, rdtype, "dresidual")
    sh = _norm_shape(dy, dtype, rdtype, 0.0)
    one = scale is None and rdtype == dtype and (dx is None or dresidual is None)
    if one:
        dx = dresidual = dx if dx is not None else dresidual if dresidual is not None else _new(dy, shape, dtype)
    else:
        dx = _new(dy, shape, dtype) if dx is None else dx
        dresidual = _new(dy, shape, rdtype) if dresidual is None else dresidual
    dweight = _new(weight, weight.shape, f32)
    dscale = None if scale is None else _new(scale, scale.shape, f32)
    ref = ctypes.byref(sh)
    workspace = _workspace(workspace, _norm_bytes(sh.rows, sh.columns, sh.groups), dy)
    _launch(index, "ssd_add_rms_norm_backward", dy.data_ptr(), _p(dresidual_out), residual_out.data_ptr(),
            weight.data_ptr(), rstd.data_ptr(), None if scale is None else x.data_ptr(), _p(scale), dx.data_ptr(),
            None if one else dresidual.data_ptr(), dweight.data_ptr(), _p(dscale), ref, workspace.data_ptr(),
            _bytes(workspace))
    return dx, dresidual, dweight, dscale


def _gated_norm_shape(x, z, weight, groups, eps, norm_before_gate):
    _shaped(x, z.shape, x.dtype, "x")
    _need(weight, x.shape[-1:], _torch().float32, "weight")
    sh = _norm_shape(x, z.dtype, x.dtype, eps, groups, norm_before_gate, _row_stride(x, "x"), _row_stride(z, "z"))
    if sh.groups != groups:
        raise ValueError("groups %r is out of range" % (groups,))
    return sh


def gated_rms_norm(x, z, weight, *, groups: int = 1, eps: float = 1e-5, norm_before_gate: bool = False, y=None,
                   want_rstd: bool = False):
    """RMS norm behind the scan with its gate: y = norm(x silu(z)) weight, or
    norm(x) weight silu(z) with ``norm_before_gate``; each of ``groups`` equal
    column ranges has its own mean.

    x [..., D] in z's dtype or fp32, z [..., D] fp32 or bf16 (each may be a
    column range of a wider tensor), weight [D] fp32.  Returns y (z's dtype),
    or (y, rstd [..., groups] fp32) with ``want_rstd``."""
    index = _gpu(x, z, weight, y)
    sh = _gated_norm_shape(x, z, weight, groups, eps, norm_before_gate)
    _need(y, x.shape, z.dtype, "y")
    if y is None:
        y = _new(x, x.shape, z.dtype)
    rstd = _new(x, x.shape[:-1] + (groups,), _torch().float32) if want_rstd else None
    _launch(index, "ssd_gated_rms_norm", x.data_ptr(), z.data_ptr(), weight.data_ptr(), y.data_ptr(), _p(rstd),
            ctypes.byref(sh))
    return (y, rstd) if want_rstd else y


def gated_rms_norm_backward(dy, x, z, weight, rstd, *, groups: int = 1, norm_before_gate: bool = False, dx=None,
                            dz=None, workspace=None):
    """Gradients of gated_rms_norm for dy (z's dtype) from its inputs and rstd:
    (dx, dz, dweight).  dx and dz may be given as column ranges of a wider
    tensor."""
    index = _gpu(x, z, dy, weight, rstd, dx, dz, workspace)
    f32 = _torch().float32
    sh = _gated_norm_shape(x, z, weight, groups, 0.0, norm_before_gate)
    _need(dy, x.shape, z.dtype, "dy")
    _need(rstd, x.shape[:-1] + (groups,), f32, "rstd")
    if dx is None:
        dx = _new(x, x.shape, x.dtype)
    if dz is None:
        dz = _new(x, x.shape, z.dtype)
    _shaped(dx, x.shape, x.dtype, "dx")
    _shaped(dz, x.shape, z.dtype, "dz")
    sh.dx_stride, sh.dz_stride = _row_stride(dx, "dx"), _row_stride(dz, "dz")
    dweight = _new(weight, weight.shape, f32)
    ref = ctypes.byref(sh)
    workspace = _workspace(workspace, _norm_bytes(sh.rows, sh.columns, sh.groups), x)
    _launch(index, "ssd_gated_rms_norm_backward", dy.data_ptr(), x.data_ptr(), z.data_ptr(), weight.data_ptr(),
            rstd.data_ptr(), dx.data_ptr(), dz.data_ptr(), dweight.data_ptr(), ref, workspace.data_ptr(),
            _bytes(workspace))
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
    dys = list(dys)
    if not 1 <= len(dys) <= 3:
        raise ValueError("%d output parts, 1 to 3 are possible" % len(dys))
    index = _gpu(x, weight, bias, cu_seqlens, conv_state, dfinal_conv_state, dx, workspace, *dys)
    f32, (C, K) = _torch().float32, (x.shape[-1], weight.shape[-1])
    _need(x, x.shape, x.dtype, "x")
    _need(weight, (C, K), f32, "weight")
    _need(bias, (C,), f32, "bias")
    sh = _ConvShape()
    keep = _sequences(sh, x, cu_seqlens, cu_seqlens_host)
    state = (sh.batch, K - 1, C)
    _need(conv_state, state, x.dtype, "conv_state")
    _need(dfinal_conv_state, state, x.dtype, "dfinal_conv_state")
    _need(dx, x.shape, x.dtype, "dx")
    sh.channels, sh.width = C, K
    sh.dtype, sh.ydtype = _code(x.dtype), _code(dys[0].dtype)
    sh.activation = 1 if activation else 0
    parts, _ = _conv_outputs(x.shape[:-1], C, [t.shape[-1] for t in dys], dys, dys[0].dtype, x.device)
    if dx is None:
        dx = _new(x, x.shape, x.dtype)
    dweight = _new(weight, weight.shape, f32)
    dbias = None if bias is None else _new(bias, bias.shape, f32)
    want = conv_state is not None if want_dstate is None else want_dstate
    dstate = _new(x, state, x.dtype) if want else None
    ref = ctypes.byref(sh)
    workspace = _workspace(workspace, _conv_bytes(sh.batch, sh.seqlen, C, K, cu_seqlens is not None), x)
    _launch(index, "ssd_causal_conv1d_backward", ctypes.byref(parts), x.data_ptr(), weight.data_ptr(), _p(bias),
            _p(conv_state), _p(dfinal_conv_state), dx.data_ptr(), dweight.data_ptr(), _p(dbias), _p(dstate), ref,
            workspace.data_ptr(), _bytes(workspace))
    del keep
    return dx, dweight, dbias, dstate
