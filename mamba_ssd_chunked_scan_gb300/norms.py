"""The norms around a block in training, and 8-bit activation checkpoints.

Wrappers over the C ABI like layer.py's: they check tensors, take device pointers and the stream, and call the
library; outputs and workspaces are allocated on the stream that the call runs on.

An 8-bit row is e4m3 codes and an fp32 scale, a power of two, and stands for codes * scale, which bf16 holds exactly.  The
forward passes leave their inputs so (``pack=True``), and the backward passes take them in place of the inputs.
"""
from __future__ import annotations

import ctypes

import torch

from .layer import (_lib, _BF16, _CODE, _E4M3, _F32, _check, _current_device, _device, _elsewhere, _empty, _lib_c, _need, _ptr, _raw_stream,
                    _real, _row_stride, _width)


def _rows_of(name, t, dtype, shape, dev):
    """Elements between the rows of a (..., width) tensor, contiguous or a column range of a wider matrix."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return shape[-1] if t.is_contiguous() else _row_stride(name, t)


def _kept(name, t, scales, scales_shape, dtype, shape, dev):
    """Check a contiguous input that may be 8-bit rows."""
    if scales is None:
        _need(name, t, dtype, shape, dev)
    else:
        _need(name, t, _E4M3, shape, dev)
        _need(name + "_scales", scales, _F32, scales_shape, dev)


def _groups(name, width, group_size):
    """How many groups of group_size columns a row has."""
    size = int(group_size)
    if size < 1 or width % size:
        raise ValueError(f"{name}: {size} does not divide the width, {width}")
    return width // size


# ---------------------------------------------------------------------------------------------- 8-bit rows

def pack_rows(x, group_size=None, *, stream=None):
    """x (..., width) bf16 or fp32 (contiguous, or a column range of a wider matrix) as 8-bit rows: (codes, scales).

    codes (..., width) float8_e4m3fn and scales fp32, (...) or, with a group_size that divides the width, (..., width /
    group_size): the smallest power of two with max |x| <= 448 * scale, at least 2^-108.  Infinities and NaNs become
    NaN by themselves.  group_size (the width, where it is not given) is at most 16384."""
    dev = _device("x", x)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return pack_rows(x, group_size)
    dtype, shape = x.dtype, x.shape
    _real("x", dtype)
    width = _width("x", shape)
    lead = shape[:-1] if group_size is None else (*shape[:-1], _groups("group_size", width, group_size))
    step = width if x.is_contiguous() else _row_stride("x", x)
    codes = _empty(shape, dtype=_E4M3, device=x.device)
    scales = _empty(lead, dtype=_F32, device=x.device)
    rc = _lib_c.ssd_pack_rows(x.numel() // width, width, width if group_size is None else int(group_size), _CODE[dtype], step, x.data_ptr(),
                              codes.data_ptr(), scales.data_ptr(), _raw_stream(dev))
    if rc:
        _check(rc, "ssd_pack_rows")
    return codes, scales


def unpack_rows(codes, scales, *, dtype=_BF16, stream=None):
    """What 8-bit rows stand for, codes * scales in fp32, in dtype (bf16 or fp32; exact for pack_rows' scales): codes (..., width) float8_e4m3fn, contiguous, and scales fp32, (...) or
    (..., groups)."""
    dev = _device("codes", codes)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return unpack_rows(codes, scales, dtype=dtype)
    _real("dtype", dtype)
    shape = codes.shape
    width = _width("codes", shape)
    _need("codes", codes, _E4M3, shape, dev)
    groups = scales.shape[-1] if scales.dim() == len(shape) else 1
    if groups < 1 or width % groups:
        raise ValueError(f"scales: {groups} groups do not divide the width, {width}")
    _need("scales", scales, _F32, (*shape[:-1], groups) if scales.dim() == len(shape) else shape[:-1], dev)
    out = _empty(shape, dtype=dtype, device=codes.device)
    rc = _lib_c.ssd_unpack_rows(codes.numel() // width, width, width // groups, _CODE[dtype], codes.data_ptr(), scales.data_ptr(),
                                out.data_ptr(), _raw_stream(dev))
    if rc:
        _check(rc, "ssd_unpack_rows")
    return out


# ---------------------------------------------------------------------------------- gate and norm after the scan

def gate_norm_pack(y, z, weight, group_size, eps=1e-5, *, stream=None):
    """gate_norm(..., pack=True)."""
    dev = _device("y", y)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return gate_norm_pack(y, z, weight, group_size, eps)
    dtype, shape, device = y.dtype, y.shape, y.device
    _real("y", dtype)
    width = _width("y", shape)
    groups = _groups("group_size", width, group_size)
    _need("y", y, dtype, shape, dev)
    zs = _rows_of("z", z, dtype, shape, dev)
    _need("weight", weight, _F32, (width,), dev)
    out = _empty(shape, dtype=dtype, device=device)
    kept = {}
    for name in ("y", "z"):
        kept[name] = _empty(shape, dtype=_E4M3, device=device)
        kept[name + "_scales"] = _empty((*shape[:-1], groups), dtype=_F32, device=device)
    p = _lib.GateNormParams(y.numel() // width, zs, width, width, width // groups, _CODE[dtype], eps)
    rc = _lib_c.ssd_gate_norm_pack(ctypes.byref(p), y.data_ptr(), z.data_ptr(), weight.data_ptr(), out.data_ptr(),
                                   *[t.data_ptr() for t in kept.values()], _raw_stream(dev))
    if rc:
        _check(rc, "ssd_gate_norm_pack")
    return out, kept


def gate_norm_bwd(dout, y, z, weight, group_size, eps=1e-5, *, y_scales=None, z_scales=None, dz=None, want_out=False, stream=None):
    """Gradients of <dout, out> of one gate_norm call.

    dout (..., width) bf16 or fp32; y and z as given to it (z may be a column range of a wider matrix), or 8-bit rows with
    y_scales, z_scales (..., width / group_size): ``gate_norm_bwd(dout, weight=w, group_size=n, **packed)`` takes what
    gate_norm(..., pack=True) left (one in 8 bits and the other not is slower).  dz may be given to be written in place, at any row stride (a column range of
    a projection's gradient, say).  Returns a dict: ``dy``, ``dz`` (dout's type), ``dweight`` (fp32) and, with want_out, ``out``: the
    call's result, computed again (else None)."""
    dev = _device("dout", dout)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return gate_norm_bwd(dout, y, z, weight, group_size, eps, y_scales=y_scales, z_scales=z_scales, dz=dz, want_out=want_out)
    dtype, shape, device = dout.dtype, dout.shape, dout.device
    _real("dout", dtype)
    width = _width("dout", shape)
    groups = _groups("group_size", width, group_size)
    _need("dout", dout, dtype, shape, dev)
    per = (*shape[:-1], groups)
    _kept("y", y, y_scales, per, dtype, shape, dev)
    if z_scales is None:
        zs = _rows_of("z", z, dtype, shape, dev)
    else:
        _kept("z", z, z_scales, per, dtype, shape, dev)
        zs = width
    _need("weight", weight, _F32, (width,), dev)
    if dz is None:
        dz, dzs = _empty(shape, dtype=dtype, device=device), width
    else:
        dzs = _rows_of("dz", dz, dtype, shape, dev)
    p = _lib.GateNormParams(dout.numel() // width, zs, dzs, width, width // groups, _CODE[dtype], eps)
    ref = ctypes.byref(p)
    nbytes = _lib_c.ssd_gate_norm_bwd_workspace_size(ref)
    dy = _empty(shape, dtype=dtype, device=device)
    out = _empty(shape, dtype=dtype, device=device) if want_out else None
    dweight = _empty(width, dtype=_F32, device=device)
    ws = _empty(nbytes, dtype=torch.uint8, device=device)
    rc = _lib_c.ssd_gate_norm_bwd(ref, dout.data_ptr(), y.data_ptr(), _ptr(y_scales), z.data_ptr(), _ptr(z_scales), weight.data_ptr(),
                                  dy.data_ptr(), dz.data_ptr(), _ptr(out), dweight.data_ptr(), ws.data_ptr(), nbytes, _raw_stream(dev))
    if rc:
        _check(rc, "ssd_gate_norm_bwd")
    return {"dy": dy, "dz": dz, "dweight": dweight, "out": out}


# ------------------------------------------------------------------------------------- the norm after a block

def _residual_type(name, dtype, rtype):
    if rtype is not _F32 and rtype is not dtype:
        raise TypeError(f"{name} must be fp32 or of x's type, got {rtype}")


def block_norm(x, weight, residual, gate=None, next_weight=None, *, scale=1.0, eps=1e-5, out_dtype=None, pack=False, stream=None):
    """The norm after a block, with the block's gate, the scaled addition to the residual stream and the next block's norm:

        u = x silu(gate) (or x);  h = residual + scale * u / sqrt(mean(u^2) + eps) * weight;
        out = h / sqrt(mean(h^2) + eps) * next_weight

    x (..., width) bf16 or fp32; residual in x's shape, fp32 (or bf16 with bf16 x); gate of x's shape and type (it may be a
    column range of a wider matrix) or None; weight, next_weight (width) fp32, next_weight None for no second norm.
    width is at most 8192.  Returns a dict: ``residual`` (h in the residual's type), ``out`` (x's type, or 8-bit rows where out_dtype is
    torch.float8_e4m3fn; None without next_weight), ``scales`` (of such rows, (...) fp32; else None), and, with pack, ``x``, ``x_scales``,
    ``gate``, ``gate_scales``: the inputs as 8-bit rows for block_norm_bwd (else None)."""
    dev = _device("x", x)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return block_norm(x, weight, residual, gate, next_weight, scale=scale, eps=eps, out_dtype=out_dtype, pack=pack)
    dtype, shape, device, rtype = x.dtype, x.shape, x.device, residual.dtype
    _real("x", dtype)
    width = _width("x", shape)
    _need("x", x, dtype, shape, dev)
    _residual_type("residual", dtype, rtype)
    _need("residual", residual, rtype, shape, dev)
    _need("weight", weight, _F32, (width,), dev)
    step = width if gate is None else _rows_of("gate", gate, dtype, shape, dev)
    if out_dtype is None:
        out_dtype = dtype
    if out_dtype is not dtype and out_dtype is not _E4M3:
        raise TypeError(f"out_dtype must be x's or float8_e4m3fn, got {out_dtype}")
    lead = shape[:-1]
    h = _empty(shape, dtype=rtype, device=device)
    out = scales = xq = xs = gq = gs = None
    if next_weight is not None:
        _need("next_weight", next_weight, _F32, (width,), dev)
        out = _empty(shape, dtype=out_dtype, device=device)
        if out_dtype is _E4M3:
            scales = _empty(lead, dtype=_F32, device=device)
    if pack:
        xq, xs = _empty(shape, dtype=_E4M3, device=device), _empty(lead, dtype=_F32, device=device)
        if gate is not None:
            gq, gs = _empty(shape, dtype=_E4M3, device=device), _empty(lead, dtype=_F32, device=device)
    p = _lib.BlockNormParams(x.numel() // width, step, width, width, _CODE[dtype], _CODE[rtype], _CODE[out_dtype], scale, eps)
    rc = _lib_c.ssd_block_norm(ctypes.byref(p), x.data_ptr(), _ptr(gate), residual.data_ptr(), weight.data_ptr(), _ptr(next_weight),
                               h.data_ptr(), _ptr(out), _ptr(scales), _ptr(xq), _ptr(xs), _ptr(gq), _ptr(gs), _raw_stream(dev))
    if rc:
        _check(rc, "ssd_block_norm")
    return {"residual": h, "out": out, "scales": scales, "x": xq, "x_scales": xs, "gate": gq, "gate_scales": gs}


def block_norm_bwd(dout, dresidual, x, h, weight, gate=None, next_weight=None, *, scale=1.0, eps=1e-5, x_scales=None, h_scales=None,
                   gate_scales=None, dgate=None, dtype=None, stream=None):
    """Gradients of <dout, out> + <dresidual, residual> of one block_norm call (out in x's type).

    dout (..., width) in dtype, bf16 or fp32 (None without next_weight); dresidual in the residual's type; x and gate as given to
    it, h its ``residual`` (not read without next_weight, and may be None then), each of them 8-bit rows where its scales (...) are
    given: the forward's with pack, or pack_rows' (one of x and gate in 8 bits and the other not is slower).  dtype is that of dout, x and gate; it need only be given where there is no dout and they are 8-bit
    rows.  dgate may be given to be written in place, at any row stride.  Returns a dict: ``dx``, ``dgate`` (None
    without a gate) in dtype, ``dresidual`` in the residual's, ``dweight`` and ``dnext_weight`` (None without
    next_weight) fp32."""
    dev = _device("dresidual", dresidual)
    if stream is not None or _current_device() != dev:
        with _elsewhere(dev, stream):
            return block_norm_bwd(dout, dresidual, x, h, weight, gate, next_weight, scale=scale, eps=eps, x_scales=x_scales, h_scales=h_scales,
                                  gate_scales=gate_scales, dgate=dgate, dtype=dtype)
    rtype, shape, device = dresidual.dtype, dresidual.shape, dresidual.device
    width = _width("dresidual", shape)
    if (dout is None) != (next_weight is None):
        raise ValueError("dout: given with next_weight, and only then")
    if h is None and (next_weight is not None or h_scales is not None):
        raise ValueError("h: given with next_weight, and with h_scales")
    if next_weight is None:
        h = h_scales = None
    if dtype is None:
        dtype = dout.dtype if dout is not None else x.dtype if x_scales is None else None
    _real("dtype", dtype)
    _residual_type("dresidual", dtype, rtype)
    _need("dresidual", dresidual, rtype, shape, dev)
    lead = shape[:-1]
    _kept("x", x, x_scales, lead, dtype, shape, dev)
    _need("weight", weight, _F32, (width,), dev)
    if next_weight is not None:
        _need("dout", dout, dtype, shape, dev)
        _kept("h", h, h_scales, lead, rtype, shape, dev)
        _need("next_weight", next_weight, _F32, (width,), dev)
    step = dstep = width
    if gate is not None:
        if gate_scales is None:
            step = _rows_of("gate", gate, dtype, shape, dev)
        else:
            _kept("gate", gate, gate_scales, lead, dtype, shape, dev)
        if dgate is None:
            dgate = _empty(shape, dtype=dtype, device=device)
        else:
            dstep = _rows_of("dgate", dgate, dtype, shape, dev)
    elif dgate is not None or gate_scales is not None:
        raise ValueError("dgate, gate_scales: only with a gate")
    p = _lib.BlockNormParams(dresidual.numel() // width, step, dstep, width, _CODE[dtype], _CODE[rtype], _CODE[dtype], scale, eps)
    ref = ctypes.byref(p)
    nbytes = _lib_c.ssd_block_norm_bwd_workspace_size(ref)
    dx = _empty(shape, dtype=dtype, device=device)
    dres = _empty(shape, dtype=rtype, device=device)
    dweight = _empty(width, dtype=_F32, device=device)
    dnext = _empty(width, dtype=_F32, device=device) if next_weight is not None else None
    ws = _empty(nbytes, dtype=torch.uint8, device=device)
    rc = _lib_c.ssd_block_norm_bwd(ref, _ptr(dout), dresidual.data_ptr(), x.data_ptr(), _ptr(x_scales), _ptr(gate), _ptr(gate_scales), _ptr(h),
                                   _ptr(h_scales), weight.data_ptr(), _ptr(next_weight), dx.data_ptr(), _ptr(dgate), dres.data_ptr(),
                                   dweight.data_ptr(), _ptr(dnext), ws.data_ptr(), nbytes, _raw_stream(dev))
    if rc:
        _check(rc, "ssd_block_norm_bwd")
    return {"dx": dx, "dgate": dgate, "dresidual": dres, "dweight": dweight, "dnext_weight": dnext}
