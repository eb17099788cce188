"""The C entry points of the operators around the scan refuse bad arguments before anything is launched
(these calls never touch the device)."""
import pytest


@pytest.fixture(scope="module")
def L():
    from mamba_ssd_chunked_scan_gb300 import build
    build.build()
    from mamba_ssd_chunked_scan_gb300 import _lib
    return _lib.lib


G = 1 << 30   # fake device addresses this far apart share no byte


def norm(L, **kw):
    d = dict(rows=16, width=256, dtype=1, rdtype=0, odtype=1, x=G, res=2 * G, w=3 * G, eps=1e-5, out=4 * G, scales=None,
             rout=5 * G, rstd=6 * G, stream=None)
    d.update(kw)
    return L.ssd_add_norm(*d.values())


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(width=0), 1), (dict(dtype=2), 1), (dict(dtype=7), 1), (dict(rdtype=2), 1),
    (dict(dtype=0, odtype=0, rdtype=1), 1), (dict(odtype=0), 1), (dict(odtype=3), 1), (dict(width=16385), 2),
    (dict(rows=1 << 31), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(x=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(odtype=2), 1),
    (dict(x=G + 1), 1), (dict(res=2 * G + 2), 1), (dict(w=3 * G + 2), 1), (dict(rstd=6 * G + 1), 1),
    (dict(out=G + 16), 1), (dict(rout=2 * G + 16), 1), (dict(out=2 * G), 1), (dict(rout=4 * G), 1), (dict(rout=G), 1),
    (dict(out=3 * G), 1), (dict(rstd=G), 1), (dict(rstd=4 * G + 8), 1), (dict(odtype=2, scales=6 * G), 1),
    (dict(odtype=2, scales=5 * G), 1),
])
def test_add_norm_refusals(L, kw, code):
    assert norm(L, **kw) == code


def norm_bwd(L, **kw):
    d = dict(rows=16, width=256, dtype=1, rdtype=0, dout=G, h=2 * G, w=3 * G, rstd=4 * G, dres=5 * G, dx=6 * G, dro=7 * G,
             dw=8 * G, ws=9 * G, wsb=1 << 28, stream=None)
    d.update(kw)
    return L.ssd_add_norm_bwd(*d.values())


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(width=0), 1), (dict(width=20000), 2), (dict(dtype=2), 1), (dict(dtype=0, rdtype=1), 1),
    (dict(dout=None), 1), (dict(h=None), 1), (dict(w=None), 1), (dict(rstd=None), 1), (dict(dw=None), 1),
    (dict(dx=None, dro=None), 1), (dict(ws=None), 3), (dict(wsb=16), 3), (dict(ws=9 * G + 4), 3), (dict(dx=2 * G), 1),
    (dict(dro=G), 1), (dict(dx=7 * G), 1), (dict(dw=6 * G), 1), (dict(dw=9 * G), 1), (dict(dx=9 * G), 1), (dict(dx=3 * G), 1),
    (dict(dro=2 * G), 1), (dict(dx=G + 16), 1), (dict(dx=6 * G + 1), 1), (dict(rows=0, dw=None), 1),
])
def test_add_norm_bwd_refusals(L, kw, code):
    assert norm_bwd(L, **kw) == code


def test_nothing_to_do(L):
    assert norm(L, rows=0, x=None, out=None) == 0
    assert L.ssd_add_norm_bwd_workspace_size(0, 64) == 0
    assert L.ssd_add_norm_bwd_workspace_size(16, 0) == 0
    assert L.ssd_add_norm_bwd_workspace_size(16, 20000) == 0
    assert L.ssd_add_norm_bwd_workspace_size(16, 256) == 16 * 256 * 4
