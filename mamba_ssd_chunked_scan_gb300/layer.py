"""The operators around the scan: residual RMS norm.

Thin wrappers over the C ABI like the package's other entry points: they check
tensors, take device pointers and the stream, and call the library.  Outputs
and workspaces are allocated on the stream that the call runs on.
"""
from __future__ import annotations

import contextlib

import torch

from . import _lib

_lib_c = _lib.lib
_BF16, _F32, _E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_CODE = {_F32: _lib.SSD_F32, _BF16: _lib.SSD_BF16, _E4M3: _lib.SSD_E4M3}


def _wrong(name, t, dtype, shape, dev):
    return ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on cuda:{dev}, got "
                      f"{t.dtype} {tuple(t.shape)} (strides {t.stride()}) on {t.device}")


def _need(name, t, dtype, shape, dev):
    """Raise unless t is a contiguous tensor of this type and shape on the device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise _wrong(name, t, dtype, shape, dev)


def _device(name, t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    return dev


@contextlib.contextmanager
def _elsewhere(dev, stream):
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


_HERE = contextlib.nullcontext()


def _on(dev, stream):
    """The context that a call's allocations and launches run in: its stream and device are the current ones."""
    if stream is None and torch.cuda.current_device() == dev:
        return _HERE
    return _elsewhere(dev, stream)


def _raw_stream(dev):
    # the current stream's handle; torch.cuda.current_stream(dev).cuda_stream builds a Stream object first,
    # several microseconds that a decoding step's call would feel
    return torch._C._cuda_getCurrentRawStream(dev)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(rc, what):
    if rc:
        raise _lib.SSDError(rc, what)


def add_norm(x, weight, residual=None, *, eps=1e-5, out_dtype=None, residual_dtype=None, return_rstd=False, stream=None):
    """Root-mean-square norm over the last dimension with the residual's addition:
    h = x + residual, out = h / sqrt(mean(h^2) + eps) * weight.

    x (..., width) bf16 or fp32; weight (width) fp32; residual in x's shape,
    fp32 (or bf16 with bf16 x), or None.  Returns a dict: ``out`` in out_dtype
    (x's dtype by default, or torch.float8_e4m3fn), ``scales`` (the shape without its last dimension, fp32; e4m3
    only: the row is out * scales), ``residual`` (h in the residual's type, or in residual_dtype where that is given
    without a residual; else None) and ``rstd`` (fp32, with return_rstd; else None)."""
    dev = _device("x", x)
    dtype, shape = x.dtype, x.shape
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError(f"x must be bf16 or fp32, got {dtype}")
    if x.dim() < 1 or shape[-1] < 1:
        raise ValueError(f"x: expected (..., width), got {tuple(shape)}")
    width = shape[-1]
    _need("x", x, dtype, shape, dev)
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
    with _on(dev, stream):
        out = torch.empty(shape, dtype=out_dtype, device=x.device)
        scales = torch.empty(shape[:-1], dtype=_F32, device=x.device) if out_dtype is _E4M3 else None
        res = None if residual_dtype is None else torch.empty(shape, dtype=residual_dtype, device=x.device)
        rstd = torch.empty(shape[:-1], dtype=_F32, device=x.device) if return_rstd else None
        rc = _lib_c.ssd_add_norm(x.numel() // width, width, _CODE[dtype], _CODE[residual_dtype or dtype], _CODE[out_dtype],
                                 x.data_ptr(), _ptr(residual), weight.data_ptr(), eps, out.data_ptr(), _ptr(scales),
                                 _ptr(res), _ptr(rstd), _raw_stream(dev))
    _check(rc, "ssd_add_norm")
    return {"out": out, "scales": scales, "residual": res, "rstd": rstd}


def add_norm_bwd(dout, h, weight, rstd, dresidual=None, *, stream=None):
    """Gradients of one add_norm call (out in x's type): dout (..., width) in x's
    type, h the call's ``residual`` (or x where it had none), rstd its ``rstd``,
    dresidual the gradient of ``residual`` in h's type, or None.  Returns a
    dict: ``dx`` (dout's type), ``dresidual`` (the same values in h's type;
    the same tensor where the types are equal) and ``dweight`` (fp32)."""
    dev = _device("dout", dout)
    dtype, rtype, shape = dout.dtype, h.dtype, dout.shape
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError(f"dout must be bf16 or fp32, got {dtype}")
    if rtype is not _F32 and rtype is not dtype:
        raise TypeError(f"h must be fp32 or of dout's type, got {rtype}")
    if dout.dim() < 1 or shape[-1] < 1:
        raise ValueError(f"dout: expected (..., width), got {tuple(shape)}")
    width = shape[-1]
    _need("dout", dout, dtype, shape, dev)
    _need("h", h, rtype, shape, dev)
    _need("weight", weight, _F32, (width,), dev)
    _need("rstd", rstd, _F32, shape[:-1], dev)
    if dresidual is not None:
        _need("dresidual", dresidual, rtype, shape, dev)
    rows = dout.numel() // width
    nbytes = _lib_c.ssd_add_norm_bwd_workspace_size(rows, width)
    with _on(dev, stream):
        dx = torch.empty_like(dout)
        dres = torch.empty_like(h) if rtype is not dtype else None
        dweight = torch.empty_like(weight)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dout.device)
        rc = _lib_c.ssd_add_norm_bwd(rows, width, _CODE[dtype], _CODE[rtype], dout.data_ptr(), h.data_ptr(),
                                     weight.data_ptr(), rstd.data_ptr(), _ptr(dresidual), dx.data_ptr(), _ptr(dres),
                                     dweight.data_ptr(), ws.data_ptr(), nbytes, _raw_stream(dev))
    _check(rc, "ssd_add_norm_bwd")
    return {"dx": dx, "dresidual": dx if dres is None else dres, "dweight": dweight}
