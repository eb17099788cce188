"""The C entry points of the norms around a block and of 8-bit rows refuse bad arguments before anything is launched (these
calls never touch the device)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def M():
    from mamba_ssd_chunked_scan_gb300 import build
    build.build()
    from mamba_ssd_chunked_scan_gb300 import _lib
    return _lib


G = 1 << 30   # fake device addresses this far apart share no byte
NAN, INF = float("nan"), float("inf")


def pack(M, **kw):
    d = dict(rows=16, width=256, group=64, dtype=1, stride=256, x=G, codes=2 * G, scales=3 * G, stream=None)
    d.update(kw)
    return M.lib.ssd_pack_rows(*d.values())


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(width=0), 1), (dict(group=0), 1), (dict(group=48), 1), (dict(dtype=2), 1), (dict(stride=255), 1), (dict(x=None), 1),
    (dict(codes=None), 1), (dict(scales=None), 1), (dict(x=G + 1), 1), (dict(scales=3 * G + 2), 1), (dict(codes=G + 100), 1), (dict(scales=2 * G + 64), 1),
    (dict(scales=G), 1), (dict(width=16385, group=16385, stride=16385), 2), (dict(stride=G), 2), (dict(rows=1 << 31), 2),
    (dict(rows=1 << 30, group=128), 2), (dict(rows=0, x=None, codes=None, scales=None), 0),
])
def test_pack_refusals(M, kw, code):
    assert pack(M, **kw) == code


def unpack(M, **kw):
    d = dict(rows=16, width=256, group=64, dtype=1, codes=G, scales=2 * G, out=3 * G, stream=None)
    d.update(kw)
    return M.lib.ssd_unpack_rows(*d.values())


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(width=0), 1), (dict(group=0), 1), (dict(group=100), 1), (dict(dtype=2), 1), (dict(codes=None), 1), (dict(scales=None), 1),
    (dict(out=None), 1), (dict(out=3 * G + 1), 1), (dict(scales=2 * G + 1), 1), (dict(out=G), 1), (dict(out=2 * G), 1), (dict(rows=1 << 31), 2),
    (dict(rows=0, out=None), 0),
])
def test_unpack_refusals(M, kw, code):
    assert unpack(M, **kw) == code


def gate_params(M, **kw):
    d = dict(rows=16, z_stride=600, dz_stride=700, width=256, group_size=128, dtype=1, eps=1e-5)
    d.update(kw)
    return M.GateNormParams(*d.values())


BAD_GATE = [(dict(rows=-1), 1), (dict(z_stride=255), 1), (dict(width=0), 1), (dict(group_size=100), 1), (dict(group_size=0), 1), (dict(dtype=2), 1),
            (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1), (dict(width=8193, group_size=8193, z_stride=8193, dz_stride=8193), 2),
            (dict(z_stride=G), 2), (dict(rows=1 << 30), 2)]


@pytest.mark.parametrize("kw,code", BAD_GATE)
def test_gate_norm_parameters(M, kw, code):
    p = gate_params(M, **kw)
    assert M.lib.ssd_gate_norm_bwd_workspace_size(p) == 0
    assert M.lib.ssd_gate_norm_pack(p, G, 2 * G, 3 * G, 4 * G, 5 * G, 6 * G, 7 * G, 8 * G, None) == code
    assert M.lib.ssd_gate_norm_bwd(p, G, 2 * G, None, 3 * G, None, 4 * G, 5 * G, 6 * G, None, 7 * G, 8 * G, 1 << 29, None) == code


def gate_pack(M, p=None, **kw):
    d = dict(y=G, z=2 * G, w=3 * G, out=4 * G, yc=5 * G, ys=6 * G, zc=7 * G, zs=8 * G, stream=None)
    d.update(kw)
    return M.lib.ssd_gate_norm_pack(p or gate_params(M), *d.values())


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, 1) for k in ("y", "z", "w", "out", "yc", "ys", "zc", "zs")],
    (dict(y=G + 1), 1), (dict(z=2 * G + 1), 1), (dict(w=3 * G + 2), 1), (dict(out=4 * G + 1), 1), (dict(ys=6 * G + 1), 1), (dict(out=G), 1),
    (dict(out=2 * G), 1), (dict(zc=5 * G), 1), (dict(zs=6 * G), 1), (dict(yc=4 * G + 8), 1), (dict(ys=3 * G), 1),
])
def test_gate_norm_pack_refusals(M, kw, code):
    assert gate_pack(M, **kw) == code


def gate_bwd(M, p=None, **kw):
    d = dict(dout=G, y=2 * G, ys=None, z=3 * G, zs=None, w=4 * G, dy=5 * G, dz=6 * G, out=7 * G, dw=8 * G, ws=9 * G, wsb=1 << 29, stream=None)
    d.update(kw)
    return M.lib.ssd_gate_norm_bwd(p or gate_params(M), *d.values())


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, 1) for k in ("dout", "y", "z", "w", "dy", "dz", "dw")],
    (dict(ws=None), 3), (dict(wsb=16), 3), (dict(ws=9 * G + 4), 3), (dict(zs=10 * G), 1), (dict(dy=G), 1), (dict(dy=2 * G), 1), (dict(dz=3 * G), 1),
    (dict(dz=5 * G), 1), (dict(out=6 * G), 1), (dict(dw=4 * G), 1), (dict(dw=9 * G), 1), (dict(ws=7 * G), 1), (dict(ys=10 * G + 2), 1), (dict(dw=8 * G + 1), 1),
    (dict(dy=5 * G + 1), 1),
])
def test_gate_norm_bwd_refusals(M, kw, code):
    assert gate_bwd(M, **kw) == code


def test_gate_norm_bwd_strides(M):
    assert gate_bwd(M, gate_params(M, dz_stride=255)) == 1
    assert gate_bwd(M, gate_params(M, dz_stride=G)) == 2


def block_params(M, **kw):
    d = dict(rows=16, gate_stride=600, dgate_stride=700, width=256, dtype=1, residual_dtype=0, out_dtype=1, scale=0.5, eps=1e-5)
    d.update(kw)
    return M.BlockNormParams(*d.values())


BAD_BLOCK = [(dict(rows=-1), 1), (dict(gate_stride=255), 1), (dict(width=0), 1), (dict(dtype=2), 1), (dict(dtype=0, residual_dtype=1, out_dtype=0), 1),
             (dict(residual_dtype=2), 1), (dict(out_dtype=0), 1), (dict(out_dtype=3), 1), (dict(scale=INF), 1), (dict(scale=NAN), 1), (dict(eps=-1.0), 1),
             (dict(eps=NAN), 1), (dict(width=8193, gate_stride=8193, dgate_stride=8193), 2), (dict(gate_stride=G), 2), (dict(rows=1 << 31), 2)]


def block(M, p=None, **kw):
    d = dict(x=G, gate=2 * G, res=3 * G, w=4 * G, w2=5 * G, h=6 * G, out=7 * G, os=None, xc=8 * G, xs=9 * G, gc=10 * G, gs=11 * G, stream=None)
    d.update(kw)
    return M.lib.ssd_block_norm(p or block_params(M), *d.values())


def block_bwd(M, p=None, **kw):
    d = dict(dout=G, dres=2 * G, x=3 * G, xs=None, gate=4 * G, gs=None, h=5 * G, hs=None, w=6 * G, w2=7 * G, dx=8 * G, dgate=9 * G, dr=10 * G,
             dw=11 * G, dw2=12 * G, ws=13 * G, wsb=1 << 29, stream=None)
    d.update(kw)
    return M.lib.ssd_block_norm_bwd(p or block_params(M), *d.values())


@pytest.mark.parametrize("kw,code", BAD_BLOCK)
def test_block_norm_parameters(M, kw, code):
    assert block(M, block_params(M, **kw)) == code
    assert block_bwd(M, block_params(M, **kw)) == code
    if "gate_stride" not in kw or kw.get("width", 0) > 8192:
        assert M.lib.ssd_block_norm_bwd_workspace_size(block_params(M, **kw)) == 0


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, 1) for k in ("x", "res", "w", "h", "out", "xc", "xs", "gc", "gs", "gate")],
    (dict(x=G + 1), 1), (dict(res=3 * G + 2), 1), (dict(w2=5 * G + 1), 1), (dict(out=G), 1), (dict(out=6 * G), 1), (dict(h=G), 1), (dict(h=3 * G + 64), 1),
    (dict(out=3 * G), 1), (dict(xc=3 * G), 1), (dict(gc=8 * G), 1), (dict(xs=7 * G), 1), (dict(gs=9 * G), 1), (dict(h=4 * G), 1),
])
def test_block_norm_refusals(M, kw, code):
    assert block(M, **kw) == code


def test_block_norm_codes_out_need_scales(M):
    assert block(M, block_params(M, out_dtype=2)) == 1
    assert block(M, block_params(M, out_dtype=2), os=7 * G) == 1


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, 1) for k in ("dout", "dres", "x", "h", "w", "w2", "dx", "dr", "dw", "dw2", "gate", "dgate")],
    (dict(ws=None), 3), (dict(wsb=64), 3), (dict(ws=13 * G + 8), 3), (dict(gs=14 * G), 1), (dict(dx=G), 1), (dict(dr=2 * G), 1), (dict(dgate=4 * G), 1),
    (dict(dx=10 * G), 1), (dict(dw=12 * G), 1), (dict(ws=8 * G), 1), (dict(dw2=7 * G), 1), (dict(hs=14 * G + 2), 1), (dict(dr=10 * G + 1), 1),
])
def test_block_norm_bwd_refusals(M, kw, code):
    assert block_bwd(M, **kw) == code


def test_workspaces_hold_every_kernel_shape(M):
    """A call's shares fit whatever its addresses and types: more rows never need less, up to the slots of the GPU."""
    for width, group in ((64, 64), (5120, 64), (2560, 2560), (2557, 2557), (8192, 8192), (8191, 8191), (264, 264), (16384, 8192)):
        sizes = [M.lib.ssd_gate_norm_bwd_workspace_size(gate_params(M, rows=r, width=width, group_size=group, z_stride=width, dz_stride=width))
                 for r in (1, 7, 100, 1000, 10000, 100000)]
        assert all(s % (4 * width) == 0 and s > 0 for s in sizes) and sizes[0] == 4 * width and sizes[1] == 28 * width
        assert max(sizes) <= 4 * width * 152 * 20 * 16 * 2
    assert M.lib.ssd_gate_norm_bwd_workspace_size(gate_params(M, rows=0)) == 0
    assert M.lib.ssd_block_norm_bwd_workspace_size(block_params(M, rows=0)) == 0
    one = M.lib.ssd_block_norm_bwd_workspace_size(block_params(M, rows=3))
    assert one == 3 * 256 * 2 * 4


def linear_packed(M, p=None, **kw):
    d = dict(x=G + 1, xs=2 * G, w=3 * G, pre=4 * G + 1, ps=5 * G, dy=6 * G, dx=7 * G, dw=8 * G, db=9 * G, ws=10 * G, wsb=1 << 29, stream=None)
    d.update(kw)
    p = p or M.LinearParams(16, 51, 24, 48, 1, 1)
    return M.lib.ssd_linear_bwd_packed(ctypes.byref(p), *d.values())


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, 1) for k in ("x", "w", "pre", "dy")],
    (dict(xs=None), 2), (dict(xs=2 * G + 2), 1), (dict(ps=5 * G + 1), 1), (dict(ps=None), 1), (dict(dx=None, dw=None, db=None), 1), (dict(dw=G), 1),
    (dict(dx=4 * G), 1), (dict(db=2 * G), 1), (dict(ws=10 * G + 16), 3), (dict(wsb=100), 3), (dict(ws=5 * G), 1), (dict(x=None, dw=None), 1),
])
def test_linear_bwd_packed_refusals(M, kw, code):
    assert linear_packed(M, **kw) == code


def test_linear_bwd_packed_parameters(M):
    for kw, code in ((dict(ldx=47), 1), (dict(k=44), 2), (dict(dtype=2), 2), (dict(ldx=G), 2), (dict(act=3), 1), (dict(n=0), 1), (dict(m=-1), 1)):
        d = dict(m=16, ldx=51, n=24, k=48, dtype=1, act=1)
        d.update(kw)
        p = M.LinearParams(*d.values())
        assert M.lib.ssd_linear_bwd_packed_workspace_size(p) == 0
        assert linear_packed(M, p) == code
    p = M.LinearParams(16, 51, 24, 48, 1, 1)
    assert M.lib.ssd_linear_bwd_packed_workspace_size(p) >= 16 * 48 * 2 + 16 * 24 * 2


def test_tensors_on_the_cpu_are_refused():
    import torch
    import mamba_ssd_chunked_scan_gb300 as ssd
    x, w = torch.zeros(4, 64), torch.ones(64)
    for bad in (lambda: ssd.pack_rows(x), lambda: ssd.unpack_rows(x.to(torch.float8_e4m3fn), w), lambda: ssd.gate_norm(x, x, w, 64, pack=True),
                lambda: ssd.gate_norm_bwd(x, x, x, w, 64), lambda: ssd.block_norm(x, w, x), lambda: ssd.block_norm_bwd(None, x, x, None, w)):
        with pytest.raises(ValueError):
            bad()
