"""The selective scan, with a decay per channel and state (``include/ssd.h``).

    y, final = selective_scan(x, dt, A, B, C, D, z, dt_softplus=True, dt_bias=bias)
    y, final, states = selective_scan(..., want_states=True)         # + selective_scan_backward
    y_t = selective_scan_step(state, x_t, dt_t, A, B_t, C_t, D, z_t, dt_softplus=True, dt_bias=bias)

In its block it follows causal_conv1d, whose step and gradients go with these.
Like the other operators these marshal arguments only, run on torch's current
stream of the tensors' device, and record no autograd graph.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Sequence

from . import SSD_F32, _DtAct, _expect, _torch
from . import block_ops as _ops
from .block_ops import _bytes, _code, _gpu, _launch, _need, _new, _p, _row_stride, _sequences, _shaped, _workspace

__all__ = ["selective_scan", "selective_scan_step", "selective_scan_backward", "SELECTIVE_STATE_ROWS"]

SELECTIVE_STATE_ROWS = 64  # SSD_SELECTIVE_STATE_ROWS of include/ssd.h


class _SelectiveShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int32),
                ("dstate", ctypes.c_int32), ("ngroups", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("ydtype", ctypes.c_int32), ("reserved", ctypes.c_int32), ("x_stride", ctypes.c_int64),
                ("dt_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64), ("b_stride", ctypes.c_int64),
                ("c_stride", ctypes.c_int64), ("dx_stride", ctypes.c_int64), ("ddt_stride", ctypes.c_int64),
                ("dz_stride", ctypes.c_int64), ("db_stride", ctypes.c_int64), ("dc_stride", ctypes.c_int64),
                ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_host", ctypes.c_void_p)]


@functools.lru_cache(maxsize=1024)
def _scan_bytes(batch, seqlen, channels, dstate, ngroups, packed, backward) -> int:
    sh = _SelectiveShape(batch, seqlen, channels, dstate, ngroups, SSD_F32, SSD_F32)
    sh.cu_seqlens = 16 if packed else None  # only whether there are offsets counts
    return _ops._query("ssd_selective_scan_workspace_size", ctypes.byref(sh), backward)


def _state_stride(t, name) -> int:
    """Elements from one row [G, N] of t to the next, 0 where the rows are dense."""
    if t.is_contiguous():
        return 0
    shape, strides = t.shape, t.stride()
    G, N = shape[-2:]
    if (N > 1 and strides[-1] != 1) or (G > 1 and strides[-2] != N):
        raise ValueError("the last two dimensions of %s must be dense" % name)
    rows, stride = 1, 0
    for n, s in zip(shape[-3::-1], strides[-3::-1]):
        if n == 1:
            continue
        if rows == 1:
            stride = s
        elif s != rows * stride:
            raise ValueError("the rows of %s are not evenly spaced" % name)
        rows *= n
    if rows > 1 and stride < G * N:
        raise ValueError("the rows of %s overlap" % name)
    return stride if rows > 1 else 0


def _activation(dt_softplus, dt_bias, dt_limit, C):
    """ssd_dt_activation by reference, or None."""
    if not dt_softplus:
        if dt_bias is not None or dt_limit is not None:
            raise ValueError("dt_bias / dt_limit need dt_softplus=True")
        return None
    _need(dt_bias, (C,), _torch().float32, "dt_bias")
    lo, hi = (0.0, math.inf) if dt_limit is None else dt_limit
    return ctypes.byref(_DtAct(_p(dt_bias), lo, hi))


def _shape(x, dt, A, B, Cm, D, z, y_dtype):
    lead, C, dtype = x.shape[:-1], x.shape[-1], x.dtype
    if B.dim() != x.dim() + 1 or A.dim() != 2:
        raise ValueError("A must be [C, N], B and C [..., G, N]")
    G, N = B.shape[-2:]
    _shaped(dt, x.shape, dtype, "dt")
    _shaped(B, lead + (G, N), dtype, "B")
    _shaped(Cm, lead + (G, N), dtype, "C")
    f32 = _torch().float32
    _need(A, (C, N), f32, "A")
    _need(D, (C,), f32, "D")
    sh = _SelectiveShape(0, 0, C, N, G, _code(dtype), _code(y_dtype), 0, _row_stride(x, "x"), _row_stride(dt, "dt"), 0,
                         _state_stride(B, "B"), _state_stride(Cm, "C"))
    if z is not None:
        _shaped(z, x.shape, dtype, "z")
        sh.z_stride = _row_stride(z, "z")
    return sh


def _states_shape(sh, packed):
    rows = SELECTIVE_STATE_ROWS
    count = sh.seqlen // rows + sh.batch if packed else sh.batch * max(-(-sh.seqlen // rows), 1)
    return count, sh.channels, sh.dstate


def selective_scan(x, dt, A, B, C, D=None, z=None, *, dt_softplus: bool = False, dt_bias=None, dt_limit=None,
                   init_state=None, cu_seqlens=None, cu_seqlens_host: Optional[Sequence[int]] = None, y=None,
                   final_state=None, want_final: bool = True, want_states: bool = False, workspace=None, y_dtype=None):
    """Selective scan over whole sequences, per channel c and state n:

        h = exp(dt A[c, n]) h + dt x B[n],   y = (sum_n h C[n] + D[c] x) silu(z)

    x, dt, z: dense [b, L, C] or packed [T, C] with ``cu_seqlens`` (int32 GPU
    tensor [b + 1]), B, C: [b, L, G, N] or [T, G, N], N at most 64, channel c in
    group c // (C // G); all of one dtype, fp32 or bf16, each may be a column
    range of a wider tensor.  A [C, N], D [C] fp32; D and z may be None (no skip,
    no gate).  ``dt_softplus``: dt holds raw step sizes and the kernels use
    ``clamp(softplus(dt + dt_bias), *dt_limit)`` (``dt_bias`` [C] fp32 or None).
    ``init_state`` [b, C, N] fp32 or None (zero).

    Returns (y, final_state), y of x's dtype unless ``y_dtype`` says fp32 or
    bf16, final_state [b, C, N] fp32 (None with ``want_final=False``); with
    ``want_states`` (y, final_state, states), the fp32 states every
    SELECTIVE_STATE_ROWS tokens that selective_scan_backward needs.

    A sequence of no tokens passes its state through.  Rows behind the last
    sequence of a packed batch are left as they were in y."""
    act_bias = dt_bias if dt_softplus else None
    index = _gpu(x, dt, A, B, C, D, z, act_bias, init_state, cu_seqlens, y, final_state, workspace)
    f32 = _torch().float32
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    sh = _shape(x, dt, A, B, C, D, z, y_dtype)
    keep = _sequences(sh, x, cu_seqlens, cu_seqlens_host)
    act = _activation(dt_softplus, dt_bias, dt_limit, sh.channels)
    state = (sh.batch, sh.channels, sh.dstate)
    _need(init_state, state, f32, "init_state")
    _need(y, x.shape, y_dtype, "y")
    _need(final_state, state, f32, "final_state")
    if y is None:
        y = _new(x, x.shape, y_dtype)
    if final_state is None and want_final:
        final_state = _new(x, state, f32)
    packed = cu_seqlens is not None
    states = _new(x, _states_shape(sh, packed), f32) if want_states else None
    need = _scan_bytes(sh.batch, sh.seqlen, sh.channels, sh.dstate, sh.ngroups, packed, 0)
    workspace = _workspace(workspace, need, x)
    _launch(index, "ssd_selective_scan", x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _p(D),
            _p(z), act, _p(init_state), y.data_ptr(), _p(final_state), _p(states), ctypes.byref(sh),
            workspace.data_ptr(), _bytes(workspace))
    del keep
    return (y, final_state, states) if want_states else (y, final_state)


def selective_scan_backward(dy, x, dt, A, B, C, states, D=None, z=None, *, dt_softplus: bool = False, dt_bias=None,
                            dt_limit=None, init_state=None, dfinal_state=None, cu_seqlens=None,
                            cu_seqlens_host: Optional[Sequence[int]] = None, dx=None, ddt=None, dB=None, dC=None,
                            dz=None, want_dinit: bool = True, dinit_state=None, workspace=None):
    """Gradients of selective_scan for dy (fp32 or bf16, shaped as x) and
    ``dfinal_state`` [b, C, N] fp32 (None: zero).  The other arguments as given to
    selective_scan, ``states`` as returned by it; they hold ``init_state``, which is
    checked and not read.

    Returns (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinit_state), ddt that of the
    raw step sizes; dD, dz and ddt_bias are None without D, z and dt_bias.  dx,
    ddt, dB, dC and dz may be given as column ranges of wider tensors.  Rows behind
    the last sequence of a packed batch are left as they were in them."""
    act_bias = dt_bias if dt_softplus else None
    index = _gpu(x, dy, dt, A, B, C, D, z, act_bias, states, init_state, dfinal_state, cu_seqlens, dx, ddt, dB, dC, dz,
                 dinit_state, workspace)
    f32 = _torch().float32
    sh = _shape(x, dt, A, B, C, D, z, dy.dtype)
    keep = _sequences(sh, x, cu_seqlens, cu_seqlens_host)
    act = _activation(dt_softplus, dt_bias, dt_limit, sh.channels)
    packed = cu_seqlens is not None
    state = (sh.batch, sh.channels, sh.dstate)
    _need(dy, x.shape, dy.dtype, "dy")
    _need(states, _states_shape(sh, packed), f32, "states")
    _need(init_state, state, f32, "init_state")
    _need(dfinal_state, state, f32, "dfinal_state")
    _need(dinit_state, state, f32, "dinit_state")
    if z is None and dz is not None:
        raise ValueError("dz without z")
    grads = {}
    for name, field, t, like, stride in (("dx", "dx_stride", dx, x, _row_stride),
                                         ("ddt", "ddt_stride", ddt, x, _row_stride),
                                         ("dB", "db_stride", dB, B, _state_stride),
                                         ("dC", "dc_stride", dC, B, _state_stride),
                                         ("dz", "dz_stride", dz, z, _row_stride)):
        if like is None:
            t = None
        elif t is None:
            t = _new(x, like.shape, x.dtype)
        else:
            _shaped(t, like.shape, x.dtype, name)
            setattr(sh, field, stride(t, name))
        grads[name] = t
    dx, ddt, dB, dC, dz = grads.values()
    dA = _new(A, A.shape, f32)
    dD = None if D is None else _new(D, D.shape, f32)
    ddt_bias = None if act_bias is None else _new(act_bias, act_bias.shape, f32)
    if dinit_state is None and want_dinit:
        dinit_state = _new(x, state, f32)
    need = _scan_bytes(sh.batch, sh.seqlen, sh.channels, sh.dstate, sh.ngroups, packed, 1)
    workspace = _workspace(workspace, need, x)
    _launch(index, "ssd_selective_scan_backward", dy.data_ptr(), _p(dfinal_state), x.data_ptr(), dt.data_ptr(),
            A.data_ptr(), B.data_ptr(), C.data_ptr(), _p(D), _p(z), act, _p(init_state), states.data_ptr(),
            dx.data_ptr(), ddt.data_ptr(), dA.data_ptr(), dB.data_ptr(), dC.data_ptr(), _p(dD), _p(dz), _p(ddt_bias),
            _p(dinit_state), ctypes.byref(sh), workspace.data_ptr(), _bytes(workspace))
    del keep
    return dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinit_state


def selective_scan_step(state, x, dt, A, B, C, D=None, z=None, *, dt_softplus: bool = False, dt_bias=None,
                        dt_limit=None, state_out=None, y=None, y_dtype=None):
    """One token per sequence: x, dt, z [b, C], B, C [b, G, N], evenly spaced rows
    (the token's slice x[:, t] of a batch); ``state`` [b, C, N] fp32 is updated in
    place, or left as it is and the new one written to ``state_out``.  The other
    arguments as for selective_scan.  Returns y [b, C], of x's dtype unless
    ``y_dtype`` says otherwise."""
    act_bias = dt_bias if dt_softplus else None
    index = _gpu(x, dt, A, B, C, D, z, act_bias, state, state_out, y)
    f32 = _torch().float32
    if x.dim() != 2:
        raise ValueError("one token per sequence: x must be [b, C]")
    if y_dtype is None:
        y_dtype = x.dtype if y is None else y.dtype
    sh = _shape(x, dt, A, B, C, D, z, y_dtype)
    sh.batch = x.shape[0]
    act = _activation(dt_softplus, dt_bias, dt_limit, sh.channels)
    whole = (sh.batch, sh.channels, sh.dstate)
    _expect(state, whole, f32, "state")
    _need(state_out, whole, f32, "state_out")
    _need(y, x.shape, y_dtype, "y")
    if y is None:
        y = _new(x, x.shape, y_dtype)
    _launch(index, "ssd_selective_scan_step", state.data_ptr(), (state if state_out is None else state_out).data_ptr(),
            x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _p(D), _p(z), act, y.data_ptr(),
            ctypes.byref(sh))
    return y
