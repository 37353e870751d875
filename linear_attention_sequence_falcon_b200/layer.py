"""The operators of the layer around a Falcon update, bound from libfalcon.so:
the gated linear recurrence (scan, scan_bwd, scan_step), the gated norm behind
a block (norm_gate, norm_gate_bwd) and the residual norm in front of one
(residual_norm, residual_norm_bwd).

Activations and their gradients share one dtype, fp32 or bf16; states, marks,
weights and the weights' gradients are fp32.  Every array is checked before a
pointer reaches the library (FalconError).  Calls enqueue on torch's current
stream of the tensors' device, or on the stream given (outputs and workspaces
made here then belong to that stream), and return without synchronising; work
that made the inputs on another stream is the caller's to wait for.  Rows are
read through a row stride where the arguments say "rows": [.., L, D] with a
contiguous last axis whose tokens lie evenly, such as half of a projection.

The small calls are bound by the host (kernels of 2-3 us), so a call whose
arrays are as they should be, on the current device, goes the short way through
_quick (csrc/quick_layer.cpp: the same checks, allocations and call in C++, half
the time), from the load of the library on.  It answers None for anything else,
and the way below is taken: it refuses with words, or handles what the short way
does not (another device or stream, arrays to write into for the norms' passes,
a workspace given).
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os

import torch

from ._lib import DTYPES, FalconError, _check, _shape_error, load, on_load

_quick = None  # the short way, where it is built and load() has loaded the library


def _bind_quick():
    """Imports the short way.  It maps libfalcon.so, so not before load() does:
    a build() in front of that would leave this process with the old kernels."""
    global _quick
    from . import build
    if not os.path.exists(build.QUICK):  # not built, or for another torch: every call goes the long way
        return
    spec = importlib.util.spec_from_file_location(__package__ + "._quick", build.QUICK)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError:  # built against something else that is gone: the same
        return
    _quick = module


on_load.append(_bind_quick)

SCAN_BLOCK = 64      # tokens between two marks of scan
NORM_MAX_D = 16384   # the longest row of the norms

_F32 = torch.float32
_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream  # torch.cuda.current_stream builds an object: 3 us a call


def _elsewhere(index, stream):
    """Whether the call has to change the current device or stream first."""
    if index < 0:
        raise FalconError("tensor is not on a CUDA device (no CPU path exists)")
    return stream is not None or index != _current_device()


def _on(t, stream):
    """Makes the tensor's device current, and the stream with it."""
    if stream is None:
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise FalconError("the stream is on %s, the tensors on %s" % (stream.device, t.device))
    return torch.cuda.stream(stream)


def _refuse(t, name, shape, dtype, index):
    if t.shape != shape:
        _shape_error("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype is not dtype:
        raise FalconError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != index:
        raise FalconError("every tensor must be on one device (%s is on %s)" % (name, t.device))
    raise FalconError("%s must be contiguous" % name)


def _need(t, name, shape, dtype, index):
    """A contiguous array of this shape, dtype and device."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        _refuse(t, name, shape, dtype, index)


def _rows(t, name, shape, dtype, index):
    """The row stride of an array of rows: contiguous last axis, the tokens of
    all its sequences evenly spaced."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        _refuse(t, name, shape, dtype, index)
    st, D = t.stride(), shape[-1]
    if st[-1] != 1 and D > 1:
        raise FalconError("the last axis of %s must be contiguous" % name)
    n, step = shape[0], st[0]  # [n, D], or [n, L, D] whose sequences follow at L rows
    if len(shape) == 3 and shape[1] > 1:
        step = st[1]
        if n > 1 and st[0] != step * shape[1]:
            raise FalconError("the rows of %s must be evenly spaced (strides %s)" % (name, st))
    elif n <= 1:
        return D
    if step < D:
        raise FalconError("the rows of %s overlap (strides %s)" % (name, st))
    return step


def _apart(t, name):
    """Refuses an array to be written whose elements share memory."""
    span = 1
    for s, n in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
        if s < span:
            raise FalconError("the elements of %s overlap (strides %s)" % (name, t.stride()))
        span = s * n


def _int_sizes(*sizes):
    for n in sizes:
        if n > 0x7FFFFFFF:
            _shape_error("a size of %d does not fit the library's int arguments" % n)


def _dtype(t, name):
    if t.dtype not in DTYPES:
        raise FalconError("%s must be fp32 or bf16, got %s" % (name, t.dtype))
    return DTYPES[t.dtype]


def _p(t):
    return None if t is None else t.data_ptr()


def _new(t, shape):
    """A new contiguous array of this shape (t's number of elements), dtype and device."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(shape)  # empty_like: 0.6 us less


def _workspace(need, workspace, like):
    if need == 0:
        return None, 0
    if workspace is None:
        return like.new_empty(need // like.element_size() + 1), need
    if workspace.device != like.device or not workspace.is_contiguous():
        raise FalconError("workspace must be a contiguous array on %s" % (like.device,))
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise FalconError("workspace of %d bytes is smaller than the %d the call needs" % (have, need))
    return workspace, have


def _eps(eps):
    eps = float(eps)
    if not eps >= 0.0:
        raise FalconError("eps must be >= 0, got %r" % eps)
    return eps


# ---------------------------------------------------------------- the gated linear recurrence

def check_scan_shapes(x, f, reset=None, initial_state=None, out=None, final_state=None, marks=None, dout=None,
                      dstate=None, dx=None, df=None):
    """Checks the arrays of scan and scan_bwd against x's [N,L,D]: f like x,
    reset [N,L] bool or uint8, states [N,D] fp32, marks
    [N,ceil(L/SCAN_BLOCK),D] fp32; x, f, dx, df are rows, the others
    contiguous.  Returns (N, L, D, row stride of x, row stride of f)."""
    if x.dim() != 3:
        _shape_error("x must be [N,L,D], got %s" % (tuple(x.shape),))
    dt = x.dtype
    _dtype(x, "x")
    shape = N, L, D = x.shape
    _int_sizes(N, L, D)
    at = x.get_device()
    ldx = _rows(x, "x", shape, dt, at)
    ldf = _rows(f, "f", shape, dt, at)
    if reset is not None:
        if reset.dtype not in (torch.bool, torch.uint8):
            raise FalconError("reset must be bool or uint8, got %s" % reset.dtype)
        _need(reset, "reset", (N, L), reset.dtype, at)
    if initial_state is not None:
        _need(initial_state, "initial_state", (N, D), _F32, at)
    if final_state is not None:
        _need(final_state, "final_state", (N, D), _F32, at)
    if dstate is not None:
        _need(dstate, "dstate", (N, D), _F32, at)
    if marks is not None:
        _need(marks, "marks", (N, -(-L // SCAN_BLOCK), D), _F32, at)
    if out is not None:
        _need(out, "out", shape, dt, at)
    if dout is not None:
        _need(dout, "dout", shape, dt, at)
    if dx is not None:
        _rows(dx, "dx", shape, dt, at)
    if df is not None:
        _rows(df, "df", shape, dt, at)
    return N, L, D, ldx, ldf


def scan(x, f, reset=None, initial_state=None, out=None, final_state=None, marks=None, want_state=True,
         want_marks=False, stream=None):
    """falcon_scan: h_t = sigmoid(f_t) h_{t-1} + (1 - sigmoid(f_t)) x_t for each
    of the D channels of N sequences, x and f [N,L,D] (rows).  Where reset
    [N,L] is set, what came before the token does not reach it (documents
    packed into one sequence).  Returns (out, final_state), and with
    want_marks the marks that scan_bwd continues from: (out, final_state,
    marks)."""
    if stream is None and _quick is not None:
        got = _quick.scan(x, f, reset, initial_state, out, final_state, marks, want_state, want_marks)
        if got is not None:
            return got if want_marks else got[:2]
    N, L, D, ldx, ldf = check_scan_shapes(x, f, reset, initial_state, out, final_state, marks)
    at = x.get_device()
    if _elsewhere(at, stream):
        with _on(x, stream):
            return scan(x, f, reset, initial_state, out, final_state, marks, want_state, want_marks)
    if out is None:
        out = _new(x, x.shape)
    if final_state is None and want_state:
        final_state = x.new_empty((N, D), dtype=_F32)
    if marks is None and want_marks:
        marks = x.new_empty((N, -(-L // SCAN_BLOCK), D), dtype=_F32)
    _check(load().falcon_scan(DTYPES[x.dtype], x.data_ptr(), f.data_ptr(), _p(reset), _p(initial_state), N, L, D, ldx,
                              ldf, out.data_ptr(), _p(final_state), _p(marks), _raw_stream(at)))
    return (out, final_state, marks) if want_marks else (out, final_state)


def scan_bwd_workspace_size(dtype, N: int, L: int, D: int, has_marks: bool) -> int:
    """falcon_scan_bwd_workspace_size: device bytes of scan_bwd's workspace."""
    n = ctypes.c_size_t(0)
    _check(load().falcon_scan_bwd_workspace_size(DTYPES[dtype], N, L, D, int(has_marks), ctypes.byref(n)))
    return int(n.value)


def scan_bwd(x, f, dout, dstate=None, reset=None, initial_state=None, marks=None, dx=None, df=None, stream=None,
             workspace=None):
    """falcon_scan_bwd_ws: the gradients of scan given dout [N,L,D] and dstate
    [N,D] fp32 (None: zero).  `marks` are those of scan with the same x, f,
    reset and initial_state; without them they are formed again first.
    Returns a dict: dx, df [N,L,D] (written into `dx`, `df` where given: rows)
    and dinitial [N,D] fp32."""
    if stream is None and _quick is not None:
        got = _quick.scan_bwd(x, f, dout, dstate, reset, initial_state, marks, dx, df, workspace)
        if got is not None:
            return {"dx": got[0], "df": got[1], "dinitial": got[2]}
    N, L, D, ldx, ldf = check_scan_shapes(x, f, reset, initial_state, None, None, marks, dout, dstate)
    at = x.get_device()
    lddx = D if dx is None else _rows(dx, "dx", x.shape, x.dtype, at)
    lddf = D if df is None else _rows(df, "df", x.shape, x.dtype, at)
    if _elsewhere(at, stream):
        with _on(x, stream):
            return scan_bwd(x, f, dout, dstate, reset, initial_state, marks, dx, df, None, workspace)
    if dx is None:
        dx = _new(x, x.shape)
    if df is None:
        df = _new(f, x.shape)
    dinitial = x.new_empty((N, D), dtype=_F32)
    ws, have = None, 0
    if marks is None:
        ws, have = _workspace(scan_bwd_workspace_size(x.dtype, N, L, D, False), workspace, x)
    _check(load().falcon_scan_bwd_ws(DTYPES[x.dtype], x.data_ptr(), f.data_ptr(), _p(reset), _p(initial_state),
                                     _p(marks), N, L, D, ldx, ldf, dout.data_ptr(), _p(dstate), dx.data_ptr(), lddx,
                                     df.data_ptr(), lddf, dinitial.data_ptr(), _p(ws), have, _raw_stream(at)))
    return {"dx": dx, "df": df, "dinitial": dinitial}


def scan_step(x, f, state, state_out=None, out=None, stream=None):
    """falcon_scan_step: one token of N sequences, x and f [N,D] (rows), state
    [N,D] fp32.  The new state is written to state_out, or over `state`
    without one.  Returns (out [N,D], the new state)."""
    if stream is None and _quick is not None:
        got = _quick.scan_step(x, f, state, state_out, out)
        if got is not None:
            return got
    if x.dim() != 2:
        _shape_error("x must be [N,D], got %s" % (tuple(x.shape),))
    dt = _dtype(x, "x")
    shape = N, D = x.shape
    _int_sizes(N, D)
    at = x.get_device()
    ldx = _rows(x, "x", shape, x.dtype, at)
    ldf = _rows(f, "f", shape, x.dtype, at)
    _need(state, "state", shape, _F32, at)
    if state_out is None:
        state_out = state
    else:
        _need(state_out, "state_out", shape, _F32, at)
    if out is not None:
        _need(out, "out", shape, x.dtype, at)
    if _elsewhere(at, stream):
        with _on(x, stream):
            return scan_step(x, f, state, state_out, out)
    if out is None:
        out = _new(x, shape)
    _check(load().falcon_scan_step(dt, x.data_ptr(), f.data_ptr(), state.data_ptr(), N, D, ldx, ldf,
                                   state_out.data_ptr(), out.data_ptr(), _raw_stream(at)))
    return out, state_out


# ---------------------------------------------------------------- the gated norm behind a block

def check_norm_gate_shapes(o, gate, weight, out=None, dout=None, do=None, dgate=None):
    """Checks the arrays of norm_gate and norm_gate_bwd against o's [B,H,L,d]
    (any strides, contiguous last axis): gate and dgate [B,L,H*d] (rows) or
    None, weight [d] or [H,d] fp32 or None, out and dout [B,L,H*d] contiguous,
    do like o.  Returns (B, H, L, d, row stride of gate)."""
    if o.dim() != 4:
        _shape_error("o must be [B,H,L,d], got %s" % (tuple(o.shape),))
    _dtype(o, "o")
    B, H, L, d = o.shape
    _int_sizes(B, H, L)
    if not 1 <= d <= NORM_MAX_D:
        _shape_error("the rows must have 1 to %d channels, got %d" % (NORM_MAX_D, d))
    dt, at, shape = o.dtype, o.get_device(), (B, L, H * d)
    if d > 1 and o.stride(3) != 1:
        raise FalconError("the last axis of o must be contiguous")
    if do is not None:
        if do.shape != o.shape or do.dtype is not dt or do.get_device() != at:
            _shape_error("do must be like o")
        if d > 1 and do.stride(3) != 1:
            raise FalconError("the last axis of do must be contiguous")
        _apart(do, "do")
    ldg = H * d
    if gate is not None:
        ldg = _rows(gate, "gate", shape, dt, at)
    if dgate is not None:
        _rows(dgate, "dgate", shape, dt, at)
    if weight is not None:
        _need(weight, "weight", (d,) if weight.dim() == 1 else (H, d), _F32, at)
    if out is not None:
        _need(out, "out", shape, dt, at)
    if dout is not None:
        _need(dout, "dout", shape, dt, at)
    return B, H, L, d, ldg


def norm_gate(o, gate, weight, eps: float, out=None, stream=None):
    """falcon_norm_gate: o [B,H,L,d] (what fwd returns, or any strides)
    divided by each row's root mean square, times weight ([d], or [H,d] for
    one per head; None: ones) and z/(1+exp(-z)) of gate [B,L,H*d] (rows; None:
    no gate).  Returns [B,L,H*d], the layout of the output projection."""
    if stream is None and _quick is not None:
        got = _quick.norm_gate(o, gate, weight, eps, out)
        if got is not None:
            return got
    B, H, L, d, ldg = check_norm_gate_shapes(o, gate, weight, out)
    eps = _eps(eps)
    at = o.get_device()
    if _elsewhere(at, stream):
        with _on(o, stream):
            return norm_gate(o, gate, weight, eps, out)
    if out is None:
        out = o.new_empty((B, L, H * d)) if gate is None else _new(gate, gate.shape)
    sb, sh, sl, _ = o.stride()
    _check(load().falcon_norm_gate(DTYPES[o.dtype], o.data_ptr(), sb, sh, sl, _p(gate), ldg, _p(weight),
                                   weight is not None and weight.dim() == 2, eps, B, H, L, d, out.data_ptr(),
                                   _raw_stream(at)))
    return out


@functools.lru_cache(maxsize=4096)
def norm_gate_bwd_workspace_size(dtype, B: int, H: int, L: int, d: int) -> int:
    """falcon_norm_gate_bwd_workspace_size: device bytes of norm_gate_bwd's workspace."""
    n = ctypes.c_size_t(0)
    _check(load().falcon_norm_gate_bwd_workspace_size(DTYPES[dtype], B, H, L, d, ctypes.byref(n)))
    return int(n.value)


def norm_gate_bwd(o, gate, weight, eps: float, dout, do=None, dgate=None, want_dweight=True, stream=None,
                  workspace=None):
    """falcon_norm_gate_bwd_ws: the gradients of norm_gate given dout
    [B,L,H*d].  Returns a dict: do [B,H,L,d] (contiguous, as bwd takes its
    dout, or written into `do` with its strides), dgate [B,L,H*d] (rows where
    given; None without a gate), dweight fp32 like weight (None without one,
    or with want_dweight=False)."""
    if stream is None and do is None and dgate is None and workspace is None and _quick is not None:
        got = _quick.norm_gate_bwd(o, gate, weight, eps, dout, want_dweight)
        if got is not None:
            return {"do": got[0], "dgate": got[1], "dweight": got[2]}
    B, H, L, d, ldg = check_norm_gate_shapes(o, gate, weight, None, dout, do)
    at = o.get_device()
    lddg = H * d
    if dgate is not None:
        if gate is None:
            raise FalconError("dgate without a gate")
        lddg = _rows(dgate, "dgate", (B, L, H * d), o.dtype, at)
    eps = _eps(eps)
    if _elsewhere(at, stream):
        with _on(o, stream):
            return norm_gate_bwd(o, gate, weight, eps, dout, do, dgate, want_dweight, None, workspace)
    if do is None:
        do = _new(o, o.shape)
    if dgate is None and gate is not None:
        dgate = _new(gate, gate.shape)
    dweight = torch.empty_like(weight) if weight is not None and want_dweight else None
    ws, have = _workspace(norm_gate_bwd_workspace_size(o.dtype, B, H, L, d), workspace, o)
    sb, sh, sl, _ = o.stride()
    tb, th, tl, _ = do.stride()
    _check(load().falcon_norm_gate_bwd_ws(DTYPES[o.dtype], o.data_ptr(), sb, sh, sl, _p(gate), ldg, _p(weight),
                                          weight is not None and weight.dim() == 2, eps, B, H, L, d, dout.data_ptr(),
                                          do.data_ptr(), tb, th, tl, _p(dgate), lddg, _p(dweight), _p(ws), have,
                                          _raw_stream(at)))
    return {"do": do, "dgate": dgate, "dweight": dweight}


# ---------------------------------------------------------------- the residual norm in front of a block

def check_residual_norm_shapes(r, weight, y=None, scale=None, **like_r):
    """Checks the arrays of residual_norm and residual_norm_bwd against r's
    [..., D]: y and every other activation like r and contiguous, scale and
    weight [D] fp32 or None.  Returns (rows, D)."""
    if r.dim() < 1:
        _shape_error("r must be [..., D]")
    _dtype(r, "r")
    shape, dt, at = r.shape, r.dtype, r.get_device()
    D = shape[-1]
    if not 1 <= D <= NORM_MAX_D:
        _shape_error("the rows must have 1 to %d channels, got %d" % (NORM_MAX_D, D))
    _need(r, "r", shape, dt, at)
    if y is not None:
        _need(y, "y", shape, dt, at)
    for name, t in like_r.items():
        if t is not None:
            _need(t, name, shape, dt, at)
    if scale is not None:
        if y is None:
            raise FalconError("a scale without what it scales (y)")
        _need(scale, "scale", (D,), _F32, at)
    if weight is not None:
        _need(weight, "weight", (D,), _F32, at)
    _int_sizes(r.numel() // D)
    return r.numel() // D, D


def residual_norm(r, weight, eps: float, y=None, scale=None, r_out=None, h=None, stream=None):
    """falcon_residual_norm: the residual stream r [..., D] plus scale [D] times
    y, and that divided by its root mean square, times weight [D].  Returns
    (r_out, h); r_out may be `r` itself (the stream updated in place), and is
    `r` where there is no y; h may be `r` or `y`, not r_out."""
    if stream is None and r_out is None and h is None and _quick is not None:
        got = _quick.residual_norm(r, weight, eps, y, scale)
        if got is not None:
            return got
    R, D = check_residual_norm_shapes(r, weight, y, scale, r_out=r_out, h=h)
    eps = _eps(eps)
    kept = r if r_out is None and y is None else r_out  # the stream that is returned, unless a new array
    if h is not None and kept is not None and h.data_ptr() == kept.data_ptr() and R:
        raise FalconError("h and r_out are the same array")
    at = r.get_device()
    if _elsewhere(at, stream):
        with _on(r, stream):
            return residual_norm(r, weight, eps, y, scale, r_out, h)
    if h is None:
        h = torch.empty_like(r)
    write = r_out
    if y is not None and r_out is None:
        write = torch.empty_like(r)
    _check(load().falcon_residual_norm(DTYPES[r.dtype], r.data_ptr(), _p(y), _p(scale), _p(weight), eps, R, D,
                                       _p(write), h.data_ptr(), _raw_stream(at)))
    return (r if write is None else write), h


@functools.lru_cache(maxsize=4096)
def residual_norm_bwd_workspace_size(dtype, R: int, D: int) -> int:
    """falcon_residual_norm_bwd_workspace_size: device bytes of residual_norm_bwd's workspace."""
    n = ctypes.c_size_t(0)
    _check(load().falcon_residual_norm_bwd_workspace_size(DTYPES[dtype], R, D, ctypes.byref(n)))
    return int(n.value)


def residual_norm_bwd(r_out, weight, eps: float, dh, dr_out=None, y=None, scale=None, dr=None, dy=None, stream=None,
                      workspace=None):
    """falcon_residual_norm_bwd_ws: the gradients of residual_norm from r_out as
    it returned it, given dh and dr_out (the gradient of r_out from what else
    reads the stream; None: zero).  Returns a dict: dr (of r), dy (of y; the
    same tensor as dr without a scale; None without y), dscale, dweight fp32
    (None without scale, weight).  dr may be dr_out or dh."""
    if stream is None and dr is None and dy is None and workspace is None and _quick is not None:
        got = _quick.residual_norm_bwd(r_out, weight, eps, dh, dr_out, y, scale)
        if got is not None:
            return {"dr": got[0], "dy": got[1], "dscale": got[2], "dweight": got[3]}
    R, D = check_residual_norm_shapes(r_out, weight, y, scale, dh=dh, dr_out=dr_out, dr=dr, dy=dy)
    eps = _eps(eps)
    if dy is not None and scale is None:
        raise FalconError("without a scale dy is dr: it is not written apart")
    if dr is not None and dy is not None and dr.data_ptr() == dy.data_ptr() and R:
        raise FalconError("dr and dy are the same array")
    at = r_out.get_device()
    if _elsewhere(at, stream):
        with _on(r_out, stream):
            return residual_norm_bwd(r_out, weight, eps, dh, dr_out, y, scale, dr, dy, None, workspace)
    if dr is None:
        dr = torch.empty_like(r_out)
    if dy is None and scale is not None:
        dy = torch.empty_like(r_out)
    dscale = None if scale is None else torch.empty_like(scale)
    dweight = None if weight is None else torch.empty_like(weight)
    ws, have = _workspace(residual_norm_bwd_workspace_size(r_out.dtype, R, D), workspace, r_out)
    _check(load().falcon_residual_norm_bwd_ws(DTYPES[r_out.dtype], r_out.data_ptr(), _p(y), _p(scale), _p(weight),
                                              dh.data_ptr(), _p(dr_out), eps, R, D, dr.data_ptr(), _p(dy), _p(dscale),
                                              _p(dweight), _p(ws), have, _raw_stream(at)))
    return {"dr": dr, "dy": dy if scale is not None else (dr if y is not None else None), "dscale": dscale,
            "dweight": dweight}
