"""Workspaces of exactly the size that is asked for, between guards: the norms' gradients by every kernel that addresses and types
choose."""
import ctypes

import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
from norms_helpers import BF, F4

pytestmark = pytest.mark.gpu

GUARD, MARK = 1 << 16, 0xA5


class Workspace:
    def __init__(self, size):
        self.size = size
        self.buffer = torch.full((GUARD + (size + 255) // 256 * 256 + GUARD,), MARK, dtype=torch.uint8, device="cuda")
        self.at = self.buffer.data_ptr() + GUARD

    def whole(self):
        return bool((self.buffer[:GUARD] == MARK).all()) and bool((self.buffer[GUARD + self.size:] == MARK).all())


def lib():
    from mamba_ssd_chunked_scan_gb300 import _lib
    return _lib


def put(t, offset):
    """t in a buffer of its own, `offset` elements in."""
    flat = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
    out = flat[offset:].view(t.shape)
    out.copy_(t)
    return out


ptr = lambda t: None if t is None else t.data_ptr()


# rows, width, groups, offset of the buffers: few rows and more than slots; lanes, CTAs, shifted vectors, single elements; late slots
SHAPES = [(1, 64, 1, 0), (7, 2560, 1, 0), (1000, 2560, 1, 0), (9733, 2560, 1, 0), (2437, 5120, 80, 0), (5003, 1533, 1, 0), (24333, 515, 1, 0), (20000, 37, 1, 0),
          (1999, 8192, 1, 0), (997, 8191, 1, 0), (3001, 520, 1, 1), (30001, 24, 1, 1), (40001, 3, 1, 0)]


@pytest.mark.parametrize("rows,width,groups,offset", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F4])
@pytest.mark.parametrize("packed", ["", "y", "yz"])
def test_gate_and_norm(rows, width, groups, offset, dtype, packed):
    L = lib()
    g = torch.Generator(device="cuda").manual_seed(rows)
    r = lambda: put(torch.randn(rows, width, generator=g, device="cuda").to(dtype), offset)
    d, t, w = r(), {"y": r(), "z": r()}, torch.rand(width, generator=g, device="cuda") + 0.5
    scales = {"y": None, "z": None}
    for name in packed:   # (rows, groups) as the forward leaves them
        t[name], scales[name] = ssd.pack_rows(t[name], width // groups)
    p = L.GateNormParams(rows, width, width, width, width // groups, 1 if dtype is BF else 0, 1e-5)
    ws = Workspace(L.lib.ssd_gate_norm_bwd_workspace_size(ctypes.byref(p)))
    dy, dz, dw = torch.empty_like(d), torch.empty_like(d), torch.empty(width, device="cuda")
    dy, dz = put(dy, offset), put(dz, offset)
    rc = L.lib.ssd_gate_norm_bwd(ctypes.byref(p), ptr(d), ptr(t["y"]), ptr(scales["y"]), ptr(t["z"]), ptr(scales["z"]), ptr(w), ptr(dy), ptr(dz), None,
                                 ptr(dw), ws.at, ws.size, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and ws.whole()
    assert dw.isfinite().all()


@pytest.mark.parametrize("rows,width,groups,offset", [s for s in SHAPES if s[2] == 1])
@pytest.mark.parametrize("dtype,rtype", [(BF, F4), (BF, BF), (F4, F4)])
@pytest.mark.parametrize("packed", ["", "x", "x gate h"])
@pytest.mark.parametrize("next_norm", [False, True])
def test_norm_after_a_block(rows, width, groups, offset, dtype, rtype, packed, next_norm):
    L = lib()
    g = torch.Generator(device="cuda").manual_seed(rows)
    r = lambda kind=dtype: put(torch.randn(rows, width, generator=g, device="cuda").to(kind), offset)
    d, dres = r(), r(rtype)
    t = {"x": r(), "gate": r(), "h": r(rtype)}
    w = torch.rand(width, generator=g, device="cuda") + 0.5
    scales = dict.fromkeys(t)
    for name in packed.split():
        t[name], scales[name] = ssd.pack_rows(t[name])
    code = lambda kind: 1 if kind is BF else 0
    p = L.BlockNormParams(rows, width, width, width, code(dtype), code(rtype), code(dtype), 0.5, 1e-5)
    ws = Workspace(L.lib.ssd_block_norm_bwd_workspace_size(ctypes.byref(p)))
    dx, dgate, dr = (put(torch.empty(rows, width, dtype=k, device="cuda"), offset) for k in (dtype, dtype, rtype))
    dw, dn = (torch.empty(width, device="cuda") for _ in range(2))
    rc = L.lib.ssd_block_norm_bwd(ctypes.byref(p), ptr(d) if next_norm else None, ptr(dres), ptr(t["x"]), ptr(scales["x"]), ptr(t["gate"]), ptr(scales["gate"]),
                                  ptr(t["h"]), ptr(scales["h"]), ptr(w), ptr(w) if next_norm else None, ptr(dx), ptr(dgate), ptr(dr), ptr(dw),
                                  ptr(dn) if next_norm else None, ws.at, ws.size, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and ws.whole()
    assert dw.isfinite().all() and (not next_norm or dn.isfinite().all())
