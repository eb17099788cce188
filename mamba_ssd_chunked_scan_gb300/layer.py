"""The operators around the scan: residual RMS norm, projection, gated recurrence.

Wrappers over the C ABI like the package's other entry points: they check
tensors, take device pointers and the stream, and call the library.  Outputs
and workspaces are allocated on the stream that the call runs on.

Device-side waits are bounded.  One that runs out (a stalled GPU) ends its kernel with outputs undefined, and offsets of
documents that break their rule leave them so too; a call with check_status=True waits for its stream and raises then, without it
nothing does.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib

_lib_c = _lib.lib
_BF16, _F32, _E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_CODE = {_F32: _lib.SSD_F32, _BF16: _lib.SSD_BF16, _E4M3: _lib.SSD_E4M3}
_ACT = {"none": 0, "silu": 1, "gelu": 2}

# The current device's number and a device's current stream's handle.  torch.cuda's functions for these check for
# initialisation and build objects first, microseconds that a decoding step's calls would feel.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_empty = torch.empty


@contextlib.contextmanager
def _elsewhere(dev, stream):
    """The given device, and stream if any, made current: a call's allocations and launches belong to them."""
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream: expected one of cuda:{dev}, where the tensors are, got one of {stream.device}")
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _device(name, t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    return dev


def _wrong(name, t, dtype, shape, dev):
    return ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on cuda:{dev}, got "
                      f"{t.dtype} {tuple(t.shape)} (strides {t.stride()}) on {t.device}")


def _need(name, t, dtype, shape, dev):
    """Raise unless t is a contiguous tensor of this type and shape on the device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise _wrong(name, t, dtype, shape, dev)


_STATUS_ONLY = 256   # a workspace that holds only the status word


def _workspace(nbytes, device, check_status):
    """A call's workspace, or None where it would hold only a status word that nobody reads."""
    if nbytes == _STATUS_ONLY and not check_status:
        return None
    return _empty(nbytes, dtype=torch.uint8, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(rc, what):
    if rc:
        raise _lib.SSDError(rc, what)


# ------------------------------------------------------------------------------------- residual RMS norm

def _real(name, dtype):
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError(f"{name} must be bf16 or fp32, got {dtype}")


def _width(name, shape):
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError(f"{name}: expected (..., width), got {tuple(shape)}")
    return shape[-1]


def add_norm(x, weight, residual=None, *, eps=1e-5, out_dtype=None, residual_dtype=None, return_rstd=False, stream=None):
    """Root-mean-square norm over the last dimension with the residual's addition:
    h = x + residual, out = h / sqrt(mean(h^2) + eps) * weight.

    x (..., width) bf16 or fp32; weight (width) fp32; residual in x's shape,
    fp32 (or bf16 with bf16 x), or None.  Returns a dict: ``out`` in out_dtype
    (x's dtype by default, or torch.float8_e4m3fn), ``scales`` (the shape without its last dimension, fp32; e4m3
    only: the row is out * scales), ``residual`` (h in the residual's type, or in residual_dtype where that is given
    without a residual; else None) and ``rstd`` (fp32, with return_rstd; else None)."""
    dev = _device("x", x)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return add_norm(x, weight, residual, eps=eps, out_dtype=out_dtype, residual_dtype=residual_dtype, return_rstd=return_rstd)
    dtype, shape, device = x.dtype, x.shape, x.device
    _real("x", dtype)
    width = _width("x", shape)
    if not x.is_contiguous():
        raise _wrong("x", x, dtype, shape, dev)
    _need("weight", weight, _F32, (width,), dev)
    if residual is not None:
        if residual_dtype is not None and residual_dtype is not residual.dtype:
            raise TypeError("residual_dtype: the residual has a type of its own")
        residual_dtype = residual.dtype
        _need("residual", residual, residual_dtype, shape, dev)
    if residual_dtype is not None and residual_dtype is not _F32 and residual_dtype is not dtype:
        raise TypeError(f"the residual must be fp32 or of x's type, got {residual_dtype}")
    if out_dtype is None:
        out_dtype = dtype
    if out_dtype is not dtype and out_dtype is not _E4M3:
        raise TypeError(f"out_dtype must be x's or float8_e4m3fn, got {out_dtype}")
    out = _empty(shape, dtype=out_dtype, device=device)
    scales = res = rstd = None
    if out_dtype is _E4M3:
        scales = _empty(shape[:-1], dtype=_F32, device=device)
    if residual_dtype is not None:
        res = _empty(shape, dtype=residual_dtype, device=device)
    if return_rstd:
        rstd = _empty(shape[:-1], dtype=_F32, device=device)
    rc = _lib_c.ssd_add_norm(x.numel() // width, width, _CODE[dtype], _CODE[residual_dtype or dtype], _CODE[out_dtype],
                             x.data_ptr(), _ptr(residual), weight.data_ptr(), eps, out.data_ptr(), _ptr(scales),
                             _ptr(res), _ptr(rstd), _raw_stream(dev))
    if rc:
        _check(rc, "ssd_add_norm")
    return {"out": out, "scales": scales, "residual": res, "rstd": rstd}


def add_norm_bwd(dout, h, weight, rstd, dresidual=None, *, stream=None):
    """Gradients of one add_norm call (out in x's type): dout (..., width) in x's
    type, h the call's ``residual`` (or x where it had none), rstd its ``rstd``,
    dresidual the gradient of ``residual`` in h's type, or None.  Returns a
    dict: ``dx`` (dout's type), ``dresidual`` (the same values in h's type;
    the same tensor where the types are equal) and ``dweight`` (fp32)."""
    dev = _device("dout", dout)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return add_norm_bwd(dout, h, weight, rstd, dresidual)
    dtype, rtype, shape, device = dout.dtype, h.dtype, dout.shape, dout.device
    _real("dout", dtype)
    if rtype is not _F32 and rtype is not dtype:
        raise TypeError(f"h must be fp32 or of dout's type, got {rtype}")
    width = _width("dout", shape)
    _need("dout", dout, dtype, shape, dev)
    _need("h", h, rtype, shape, dev)
    _need("weight", weight, _F32, (width,), dev)
    _need("rstd", rstd, _F32, shape[:-1], dev)
    if dresidual is not None:
        _need("dresidual", dresidual, rtype, shape, dev)
    rows = dout.numel() // width
    nbytes = _lib_c.ssd_add_norm_bwd_workspace_size(rows, width)
    dx = _empty(shape, dtype=dtype, device=device)
    dres = _empty(shape, dtype=rtype, device=device) if rtype is not dtype else None
    dweight = _empty(width, dtype=_F32, device=device)
    ws = _empty(nbytes, dtype=torch.uint8, device=device)
    rc = _lib_c.ssd_add_norm_bwd(rows, width, _CODE[dtype], _CODE[rtype], dout.data_ptr(), h.data_ptr(),
                                 weight.data_ptr(), rstd.data_ptr(), _ptr(dresidual), dx.data_ptr(), _ptr(dres),
                                 dweight.data_ptr(), ws.data_ptr(), nbytes, _raw_stream(dev))
    if rc:
        _check(rc, "ssd_add_norm_bwd")
    return {"dx": dx, "dresidual": dx if dres is None else dres, "dweight": dweight}


# --------------------------------------------------------------------------------------------- projection

def _row_stride(name, t):
    """Elements between the rows of a (..., k) tensor whose rows lie at one stride (its length where there is one row);
    the strides of dimensions of one say nothing."""
    st, shape = t.stride(), t.shape
    ok = len(shape) > 1 and (st[-1] == 1 or shape[-1] == 1)
    step, rows = shape[-1], 1
    for k in range(len(shape) - 2, -1, -1):
        if shape[k] == 1:
            continue
        if rows == 1:
            step = st[k]
        ok = ok and st[k] == step * rows
        rows *= shape[k]
    if not ok or step < shape[-1]:
        raise ValueError(f"{name}: expected columns together and rows at one stride, got strides {st} for {tuple(shape)}")
    return step


def _linear_params(x, w, act, dev):
    """(rows' shape, parameters) of a product x w^T."""
    dtype, shape, wshape = x.dtype, x.shape, w.shape
    if dtype is not _BF16 and dtype is not _E4M3:
        raise TypeError(f"x must be bf16 or float8_e4m3fn, got {dtype}")
    if len(shape) < 1 or len(wshape) != 2 or wshape[1] != shape[-1]:
        raise ValueError(f"expected x (..., k) and w (n, k), got {tuple(shape)} and {tuple(wshape)}")
    code = _ACT.get(act)
    if code is None:
        raise ValueError(f"act must be one of {tuple(_ACT)}, got {act!r}")
    n, k = wshape
    _need("w", w, dtype, wshape, dev)
    ldx = k if x.is_contiguous() else _row_stride("x", x)
    return shape[:-1], _lib.LinearParams(x.numel() // k if k else 0, ldx, n, k, _CODE[dtype], code)


def linear(x, w, bias=None, residual=None, *, act="none", x_scales=None, w_scales=None, return_pre=False,
           check_status=False, stream=None):
    """y = act(x w^T + bias) + residual in one product on the tensor cores.

    x (..., k) bf16, or float8_e4m3fn with x_scales (...) and w_scales (n) fp32
    (add_norm's ``out`` and ``scales``, say); rows may be column ranges of a wider matrix. w (n, k) of
    x's type; bias (n) fp32 or None; residual (..., n) bf16 or None; act "none", "silu" or "gelu" (tanh form).
    k is a multiple of 8 (bf16) or 16 (e4m3).  Returns y (..., n) bf16, or (y, pre) with return_pre: pre is the
    activation's argument in bf16, for linear_bwd.  With check_status, also synchronises the stream and raises if a
    device-side wait ran out."""
    dev = _device("x", x)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return linear(x, w, bias, residual, act=act, x_scales=x_scales, w_scales=w_scales, return_pre=return_pre,
                          check_status=check_status)
    lead, p = _linear_params(x, w, act, dev)
    n, device = p.n, x.device
    if x.dtype is _E4M3:
        if x_scales is None or w_scales is None:
            raise ValueError("x_scales, w_scales: e4m3 operands come with both")
        _need("x_scales", x_scales, _F32, lead, dev)
        _need("w_scales", w_scales, _F32, (n,), dev)
    elif x_scales is not None or w_scales is not None:
        raise ValueError("x_scales, w_scales: only with e4m3 operands")
    if bias is not None:
        _need("bias", bias, _F32, (n,), dev)
    out_shape = (*lead, n)
    if residual is not None:
        _need("residual", residual, _BF16, out_shape, dev)
    ref = ctypes.byref(p)
    nbytes = _lib_c.ssd_linear_workspace_size(ref)
    if nbytes == 0:
        raise _lib.SSDError(2, f"linear of {tuple(x.shape)} and {tuple(w.shape)}, row stride {p.ldx}")
    y = _empty(out_shape, dtype=_BF16, device=device)
    pre = _empty(out_shape, dtype=_BF16, device=device) if return_pre else None
    ws = _workspace(nbytes, device, check_status)
    st = _raw_stream(dev)
    rc = _lib_c.ssd_linear(ref, x.data_ptr(), w.data_ptr(), _ptr(x_scales), _ptr(w_scales), _ptr(bias), _ptr(residual),
                           y.data_ptr(), _ptr(pre), _ptr(ws), nbytes, st)
    if rc:
        _check(rc, "ssd_linear")
    if check_status and p.m:
        _check(_lib_c.ssd_check_status(ws.data_ptr(), st), "ssd_linear device status")
    return (y, pre) if return_pre else y


def linear_bwd(dy, x, w, pre=None, *, act="none", want_dx=True, want_dw=True, want_dbias=False, check_status=False, stream=None):
    """Gradients of <dy, y> of one linear call of bf16 operands: dy (..., n) bf16, x and w as given to it, pre
    its second result (with an activation).  Returns a dict: ``dx`` (..., k) bf16, ``dw`` (n, k) bf16 and
    ``dbias`` (n) fp32, None where not wanted.  (The residual's gradient is dy.)"""
    dev = _device("x", x)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return linear_bwd(dy, x, w, pre, act=act, want_dx=want_dx, want_dw=want_dw, want_dbias=want_dbias, check_status=check_status)
    lead, p = _linear_params(x, w, act, dev)
    device = x.device
    if x.dtype is not _BF16:
        raise TypeError(f"x must be bf16, got {x.dtype}")
    out_shape = (*lead, p.n)
    _need("dy", dy, _BF16, out_shape, dev)
    if (pre is None) != (act == "none"):
        raise ValueError("pre: given with an activation, and only then")
    if pre is not None:
        _need("pre", pre, _BF16, out_shape, dev)
    if not (want_dx or want_dw or want_dbias):
        raise ValueError("no gradient wanted")
    ref = ctypes.byref(p)
    nbytes = _lib_c.ssd_linear_bwd_workspace_size(ref)
    if nbytes == 0:
        raise _lib.SSDError(2, f"linear_bwd of {tuple(x.shape)} and {tuple(w.shape)}, row stride {p.ldx}")
    dx = _empty((*lead, p.k), dtype=_BF16, device=device) if want_dx else None
    dw = _empty((p.n, p.k), dtype=_BF16, device=device) if want_dw else None
    db = _empty(p.n, dtype=_F32, device=device) if want_dbias else None
    ws = _empty(nbytes, dtype=torch.uint8, device=device)
    st = _raw_stream(dev)
    rc = _lib_c.ssd_linear_bwd(ref, x.data_ptr(), w.data_ptr(), _ptr(pre), dy.data_ptr(), _ptr(dx), _ptr(dw), _ptr(db),
                               ws.data_ptr(), nbytes, st)
    if rc:
        _check(rc, "ssd_linear_bwd")
    if check_status and p.m:
        _check(_lib_c.ssd_check_status(ws.data_ptr(), st), "ssd_linear_bwd device status")
    return {"dx": dx, "dw": dw, "dbias": db}


# -------------------------------------------------------------------------------------- gated recurrence

def _token_stride(name, t, dtype, shape, dev):
    """Elements between the tokens of a (..., width) tensor whose rows may be column ranges of a wider
    matrix: the channels lie together and the leading dimensions are packed."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        raise _wrong(name, t, dtype, shape, dev)
    return shape[-1] if t.is_contiguous() else _row_stride(name, t)


def _scan_args(g, x, initial_states, cu_seqlens, dev):
    dtype, shape = g.dtype, g.shape
    _real("g", dtype)
    if len(shape) != 3:
        raise ValueError(f"g: expected (batch, seqlen, width), got {tuple(shape)}")
    batch, seqlen, width = shape
    ndocs = 0
    if cu_seqlens is not None:
        if cu_seqlens.dtype is not torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or \
                cu_seqlens.get_device() != dev or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens: expected int32 (ndocs + 1) on the device")
        ndocs = cu_seqlens.numel() - 1
    p = _lib.GateScanParams(batch, seqlen, _token_stride("g", g, dtype, shape, dev), _token_stride("x", x, dtype, shape, dev),
                            width, ndocs, _CODE[dtype])
    states = (ndocs or batch, width)
    if initial_states is not None:
        _need("initial_states", initial_states, _F32, states, dev)
    ref = ctypes.byref(p)
    nbytes = _lib_c.ssd_gate_scan_workspace_size(ref)
    if nbytes == 0:
        raise _lib.SSDError(1, f"gate scan of {tuple(shape)} with {ndocs} documents")
    return p, ref, states, nbytes


def gate_scan(g, x, initial_states=None, cu_seqlens=None, *, return_final_states=False, check_status=False, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t with a = sigmoid(g), one decay per channel and token.

    g, x (batch, seqlen, width) bf16 or fp32, contiguous or column ranges of a
    wider matrix; initial_states (batch or ndocs, width) fp32 or None;
    cu_seqlens (ndocs + 1) int32 or None (batch 1).  Returns y (g's type), or
    (y, final_states) when asked.  With check_status, also synchronises the stream and raises if the
    device recorded an error (offsets that are not increasing from 0 to seqlen)."""
    dev = _device("g", g)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return gate_scan(g, x, initial_states, cu_seqlens, return_final_states=return_final_states, check_status=check_status)
    p, ref, states, nbytes = _scan_args(g, x, initial_states, cu_seqlens, dev)
    device = g.device
    y = _empty(g.shape, dtype=g.dtype, device=device)
    fin = _empty(states, dtype=_F32, device=device) if return_final_states else None
    ws = _workspace(nbytes, device, check_status)
    st = _raw_stream(dev)
    rc = _lib_c.ssd_gate_scan(ref, g.data_ptr(), x.data_ptr(), _ptr(initial_states), _ptr(cu_seqlens), y.data_ptr(), _ptr(fin),
                              _ptr(ws), nbytes, st)
    if rc:
        _check(rc, "ssd_gate_scan")
    if check_status:
        _check(_lib_c.ssd_check_status(ws.data_ptr(), st), "ssd_gate_scan device status")
    return (y, fin) if return_final_states else y


def _like_rows(t, step):
    """An uninitialised tensor of t's shape with `step` elements between tokens."""
    if step == t.shape[-1]:
        return _empty(t.shape, dtype=t.dtype, device=t.device)
    return _empty((*t.shape[:-1], step), dtype=t.dtype, device=t.device)[..., : t.shape[-1]]


def gate_scan_bwd(g, x, y, dy, initial_states=None, dfinal_states=None, cu_seqlens=None, *, want_dinit=None, dg=None,
                  dx=None, check_status=False, stream=None):
    """Gradients of <dy, y> + <dfinal_states, final_states> of one gate_scan call, whose output was y.

    dg and dx may be given to be written in place: of g's and x's shapes and token strides (column ranges of a
    projection's gradient, say); by default they are allocated with these strides.
    Returns a dict with dg, dx and dinit (None unless want_dinit; by default with initial_states).  States inside are recomputed
    from y's every few tokens: with bf16 the difference of state and input in dg keeps y's rounding, 2^-9 of the state."""
    dev = _device("g", g)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return gate_scan_bwd(g, x, y, dy, initial_states, dfinal_states, cu_seqlens, want_dinit=want_dinit, dg=dg, dx=dx,
                                 check_status=check_status)
    p, ref, states, nbytes = _scan_args(g, x, initial_states, cu_seqlens, dev)
    dtype, shape = g.dtype, g.shape
    _need("y", y, dtype, shape, dev)
    _need("dy", dy, dtype, shape, dev)
    if dfinal_states is not None:
        _need("dfinal_states", dfinal_states, _F32, states, dev)
    if want_dinit is None:
        want_dinit = initial_states is not None
    for name, t, step in (("dg", dg, p.g_stride), ("dx", dx, p.x_stride)):
        if t is not None and _token_stride(name, t, dtype, shape, dev) != step:
            raise ValueError(f"{name}: expected the token stride of {name[1:]}, {step}")
    if dg is None:
        dg = _like_rows(g, p.g_stride)
    if dx is None:
        dx = _like_rows(x, p.x_stride)
    dinit = _empty(states, dtype=_F32, device=g.device) if want_dinit else None
    ws = _workspace(nbytes, g.device, check_status)
    st = _raw_stream(dev)
    rc = _lib_c.ssd_gate_scan_bwd(ref, g.data_ptr(), x.data_ptr(), y.data_ptr(), _ptr(initial_states), _ptr(cu_seqlens),
                                  dy.data_ptr(), _ptr(dfinal_states), dg.data_ptr(), dx.data_ptr(), _ptr(dinit), _ptr(ws),
                                  nbytes, st)
    if rc:
        _check(rc, "ssd_gate_scan_bwd")
    if check_status:
        _check(_lib_c.ssd_check_status(ws.data_ptr(), st), "ssd_gate_scan_bwd device status")
    return {"dg": dg, "dx": dx, "dinit": dinit}


def gate_scan_step(state, g, x, *, state_out=None, stream=None):
    """One token per row of the gated recurrence: state (batch, width) fp32 is
    updated in place unless state_out is given; g, x (batch, width) bf16 or
    fp32 (rows may be column ranges).  Returns y (batch, width) in g's type."""
    dev = _device("g", g)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return gate_scan_step(state, g, x, state_out=state_out)
    dtype, shape = g.dtype, g.shape
    _real("g", dtype)
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"g: expected (batch, width), got {tuple(shape)}")
    gs, xs = _token_stride("g", g, dtype, shape, dev), _token_stride("x", x, dtype, shape, dev)
    _need("state", state, _F32, shape, dev)
    if state_out is None:
        state_out = state
    else:
        _need("state_out", state_out, _F32, shape, dev)
    y = _empty(shape, dtype=dtype, device=g.device)
    rc = _lib_c.ssd_gate_scan_step(shape[0], shape[1], _CODE[dtype], gs, xs, g.data_ptr(), x.data_ptr(),
                                   state.data_ptr(), state_out.data_ptr(), y.data_ptr(), _raw_stream(dev))
    if rc:
        _check(rc, "ssd_gate_scan_step")
    return y
