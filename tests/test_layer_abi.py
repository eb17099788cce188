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


def scan_params(**kw):
    from mamba_ssd_chunked_scan_gb300 import _lib
    d = dict(batch=2, seqlen=1000, g_stride=256, x_stride=256, width=128, ndocs=0, dtype=1)
    d.update(kw)
    return _lib.GateScanParams(*d.values())


SCAN_PARAMS = [
    (dict(batch=0), 1), (dict(seqlen=0), 1), (dict(width=0), 1), (dict(g_stride=127), 1), (dict(x_stride=0), 1),
    (dict(dtype=2), 1), (dict(ndocs=-1), 1), (dict(ndocs=2), 1), (dict(seqlen=1 << 31), 2), (dict(batch=1 << 31), 2),
    (dict(g_stride=1 << 31), 2), (dict(g_stride=1 << 29), 2), (dict(batch=1 << 20, seqlen=1 << 20, width=4096, g_stride=4096, x_stride=4096), 2),
]


@pytest.mark.parametrize("kw,code", SCAN_PARAMS)
def test_gate_scan_parameters(L, kw, code):
    p = scan_params(**kw)
    assert L.ssd_gate_scan_workspace_size(p) == 0
    assert L.ssd_gate_scan(p, G, 2 * G, None, None, 3 * G, None, 4 * G, 1 << 28, None) == code
    assert L.ssd_gate_scan_bwd(p, G, 2 * G, 3 * G, None, None, 4 * G, None, 5 * G, 6 * G, None, 7 * G, 1 << 28, None) == code


def scan(L, p=None, **kw):
    d = dict(g=G, x=G + 256, init=2 * G, cu=None, y=3 * G, fin=4 * G, ws=5 * G, wsb=1 << 28, stream=None)
    d.update(kw)
    return L.ssd_gate_scan(p or scan_params(), *d.values())


@pytest.mark.parametrize("kw,code", [
    (dict(g=None), 1), (dict(x=None), 1), (dict(y=None), 1), (dict(cu=6 * G), 1), (dict(g=G + 1), 1), (dict(fin=4 * G + 2), 1),
    (dict(ws=None), 3), (dict(wsb=100), 3), (dict(ws=5 * G + 16), 3), (dict(y=G), 1), (dict(y=G + 256), 1), (dict(fin=2 * G), 1),
    (dict(fin=3 * G + 64), 1), (dict(y=5 * G + 64), 1), (dict(fin=2 * G + 512), 1),
])
def test_gate_scan_refusals(L, kw, code):
    assert scan(L, **kw) == code


def test_gate_scan_refuses_documents_without_offsets(L):
    assert scan(L, scan_params(batch=1, ndocs=3)) == 1


def scan_bwd(L, **kw):
    # dg and dx: the two halves of one matrix
    d = dict(g=G, x=G + 256, y=2 * G, init=3 * G, cu=None, dy=4 * G, dfin=5 * G, dg=6 * G, dx=6 * G + 256, dinit=7 * G, ws=8 * G,
             wsb=1 << 28, stream=None)
    d.update(kw)
    return L.ssd_gate_scan_bwd(scan_params(), *d.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), 1), (dict(y=None), 1), (dict(dg=None), 1), (dict(dx=None), 1), (dict(dx=6 * G + 128), 1), (dict(dx=6 * G + 384), 1),
    (dict(dg=G), 1), (dict(dx=4 * G), 1), (dict(dinit=5 * G), 1), (dict(ws=8 * G + 8), 3), (dict(wsb=0), 3), (dict(dinit=8 * G), 1),
])
def test_gate_scan_bwd_refusals(L, kw, code):
    assert scan_bwd(L, **kw) == code


def step(L, **kw):
    d = dict(batch=4, width=128, dtype=1, gs=256, xs=256, g=G, x=G + 256, si=2 * G, so=2 * G, y=3 * G, stream=None)
    d.update(kw)
    return L.ssd_gate_scan_step(*d.values())


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 1), (dict(width=0), 1), (dict(dtype=2), 1), (dict(gs=100), 1), (dict(g=None), 1), (dict(y=None), 1),
    (dict(si=None), 1), (dict(so=2 * G + 4), 1), (dict(y=2 * G), 1), (dict(y=G), 1), (dict(so=G), 1), (dict(x=G + 257), 1),
    (dict(batch=1 << 36), 2), (dict(batch=0), 0),
])
def test_gate_scan_step_refusals(L, kw, code):
    assert step(L, **kw) == code


def linear_params(**kw):
    from mamba_ssd_chunked_scan_gb300 import _lib
    d = dict(m=32, ldx=256, n=512, k=256, dtype=1, act=0)
    d.update(kw)
    return _lib.LinearParams(*d.values())


LINEAR_PARAMS = [
    (dict(m=-1), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(ldx=248), 1), (dict(dtype=0), 1), (dict(dtype=5), 1), (dict(act=3), 1),
    (dict(act=-1), 1), (dict(k=252), 2), (dict(ldx=260), 2), (dict(dtype=2, k=248), 2), (dict(m=1 << 30), 2),
    (dict(m=1 << 29, n=1 << 29), 2), (dict(ldx=1 << 31), 2),
]


@pytest.mark.parametrize("kw,code", LINEAR_PARAMS)
def test_linear_parameters(L, kw, code):
    p = linear_params(**kw)
    assert L.ssd_linear_workspace_size(p) == 0 and L.ssd_linear_bwd_workspace_size(p) == 0
    assert L.ssd_linear(p, G, 2 * G, None, None, None, None, 3 * G, None, 4 * G, 1 << 29, None) == code
    if kw.get("dtype") != 2:
        assert L.ssd_linear_bwd(p, G, 2 * G, None, 3 * G, 4 * G, 5 * G, None, 6 * G, 1 << 29, None) == code


def lin(L, p=None, **kw):
    d = dict(x=G, w=2 * G, xs=None, ws=None, bias=3 * G, res=4 * G, y=5 * G, pre=6 * G, work=7 * G, wb=1 << 29, stream=None)
    d.update(kw)
    return L.ssd_linear(p or linear_params(), *d.values())


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(x=G + 8), 1), (dict(w=2 * G + 2), 1), (dict(bias=3 * G + 2), 1),
    (dict(y=5 * G + 1), 1), (dict(xs=8 * G), 1), (dict(xs=8 * G, ws=9 * G), 1), (dict(wb=64), 3),
    (dict(work=7 * G + 16), 3), (dict(y=G), 1), (dict(y=2 * G + 2), 1), (dict(y=6 * G), 1), (dict(pre=4 * G), 1), (dict(y=4 * G + 2), 1),
    (dict(y=7 * G), 1), (dict(pre=3 * G), 1), (dict(res=7 * G), 1),
])
def test_linear_refusals(L, kw, code):
    assert lin(L, **kw) == code


def test_linear_workspace_missing(L):
    """Only a workspace that would hold no more than the status word may be left out (this product's parts need one)."""
    p = linear_params(m=8, n=2560, k=5120, ldx=5120)
    assert L.ssd_linear_workspace_size(p) > 256
    assert lin(L, p, work=None) == 3
    assert L.ssd_linear_workspace_size(linear_params()) == 256


def test_linear_scales_come_with_e4m3(L):
    p = linear_params(dtype=2)
    assert lin(L, p) == 1 and lin(L, p, xs=8 * G) == 1 and lin(L, p, ws=9 * G) == 1
    assert lin(L, p, xs=8 * G, ws=9 * G, y=8 * G) == 1
    assert lin(L, linear_params(m=0), x=None, y=None) == 0
    assert L.ssd_linear_bwd(p, G, 2 * G, None, 3 * G, 4 * G, 5 * G, None, 6 * G, 1 << 29, None) == 2


def lin_bwd(L, act=1, **kw):
    d = dict(x=G, w=2 * G, pre=3 * G, dy=4 * G, dx=5 * G, dw=6 * G, db=7 * G, work=8 * G, wb=1 << 29, stream=None)
    d.update(kw)
    return L.ssd_linear_bwd(linear_params(act=act), *d.values())


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(dy=None), 1), (dict(pre=None), 1), (dict(act=0), 1), (dict(dx=None, dw=None, db=None), 1),
    (dict(dy=4 * G + 8), 1), (dict(db=7 * G + 2), 1), (dict(dx=G), 1), (dict(dw=2 * G), 1), (dict(dx=4 * G + 64), 1), (dict(dw=5 * G), 1),
    (dict(db=6 * G), 1), (dict(dx=8 * G), 1), (dict(work=None), 3), (dict(wb=256), 3), (dict(work=8 * G + 128), 3),
])
def test_linear_bwd_refusals(L, kw, code):
    assert lin_bwd(L, **kw) == code


def test_linear_workspaces_hold_few_parts(L):
    """The parts of split contractions are those of one wave of tiles at most: 16 of 152 tiles of 128 x 256 sums."""
    for m in (1, 8, 64, 65, 128, 500, 4099, 16384):
        for n in (1, 33, 512, 2560, 10240):
            for k in (16, 64, 512, 2560, 5120):
                size = L.ssd_linear_workspace_size(linear_params(m=m, n=n, k=k, ldx=k))
                assert 256 <= size <= 256 + 16 * 152 * 128 * 256 * 4
                if k * 2 <= 4 * 128:
                    assert size == 256   # too short to split


def test_linear_plan_query(L):
    from mamba_ssd_chunked_scan_gb300 import _lib
    out = _lib.LinearPlan()
    p = linear_params()
    for kw, code in LINEAR_PARAMS:
        assert L.ssd_linear_plan(linear_params(**kw), 0, out) == code
    assert L.ssd_linear_plan(p, 3, out) == 1 and L.ssd_linear_plan(p, -1, out) == 1 and L.ssd_linear_plan(p, 0, None) == 1
    assert L.ssd_linear_plan(linear_params(dtype=2), 1, out) == 2 and L.ssd_linear_plan(linear_params(dtype=2), 0, out) == 0
    assert L.ssd_linear_plan(linear_params(m=0), 0, out) == 0 and out.tiles == 0
    # the workspace is the status word and the parts
    for m, n, k in ((8, 2560, 5120), (292, 6412, 3920), (4099, 2560, 5120), (300, 520, 256)):
        q = _lib.linear_plan(m, n, k, 1)
        parts = (q.tiles - q.whole) * q.splits if q.splits > 1 else 0
        assert L.ssd_linear_workspace_size(linear_params(m=m, n=n, k=k, ldx=k)) == 256 + 4 * parts * q.tile_rows * q.tile_cols


def test_fault_injection_refusals(L):
    """An injected stall wants a workspace (its status word), a count of loads and a cap that the drains outlast."""
    p, q = linear_params(), scan_params()
    lin_args = [p, G, 2 * G, None, None, None, None, 3 * G, None]
    scan_args = [q, G, G + 256, None, None, 3 * G, None]
    for loads, rounds, code in ((-1, 1 << 14, 1), (0, 4095, 1), (0, 0, 1)):
        assert L.ssd_linear_fault_inject(*lin_args, 4 * G, 1 << 29, loads, rounds, None) == code
    for loads, rounds, code in ((-2, 1 << 14, 1), (0, 4095, 1), (-1, 0, 1)):
        assert L.ssd_gate_scan_fault_inject(*scan_args, 4 * G, 1 << 28, loads, rounds, None) == code
    assert L.ssd_linear_fault_inject(*lin_args, None, 0, 0, 1 << 14, None) == 3
    assert L.ssd_gate_scan_fault_inject(*scan_args, None, 0, 0, 1 << 14, None) == 3
    assert L.ssd_linear_fault_inject(linear_params(k=0), *lin_args[1:], 4 * G, 1 << 29, 0, 1 << 14, None) == 1
    assert L.ssd_gate_scan_fault_inject(scan_params(width=0), *scan_args[1:], 4 * G, 1 << 28, 0, 1 << 14, None) == 1
