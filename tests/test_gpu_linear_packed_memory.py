"""A projection's gradients where no codes of x are expanded: x not there, in bf16, or not read since dw is not wanted.  The workspace
is then linear_bwd's, without room for x in bf16."""
import ctypes

import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
from norms_helpers import BF, E4

pytestmark = pytest.mark.gpu

M, N, K = 1000, 640, 1288


def make(seed, m=M, n=N, k=K):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    x, w, dy = r(m, k), r(n, k), r(m, n)
    return x, w, dy, ssd.pack_rows(r(m, n))


@pytest.mark.parametrize("which", ["no x", "codes of x that are not read", "x in bf16"])
def test_a_plain_workspace_is_enough(which):
    from mamba_ssd_chunked_scan_gb300 import _lib as L
    x, w, dy, (pre, ps) = make(1)
    xq, xs = ssd.pack_rows(x)
    p = L.LinearParams(M, K, N, K, 1, 1)
    size = L.lib.ssd_linear_bwd_workspace_size(ctypes.byref(p))
    assert size + 2 * M * K <= L.lib.ssd_linear_bwd_packed_workspace_size(ctypes.byref(p))
    ws = torch.full((size + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 256 == 0
    dx, dw, db = torch.empty(M, K, dtype=BF, device="cuda"), torch.empty(N, K, dtype=BF, device="cuda"), torch.empty(N, device="cuda")
    px, pxs = {"no x": (None, None), "codes of x that are not read": (xq.data_ptr(), xs.data_ptr()), "x in bf16": (x.data_ptr(), None)}[which]
    want_dw = which == "x in bf16"
    rc = L.lib.ssd_linear_bwd_packed(ctypes.byref(p), px, pxs, w.data_ptr(), pre.data_ptr(), ps.data_ptr(), dy.data_ptr(), dx.data_ptr(),
                                     dw.data_ptr() if want_dw else None, db.data_ptr(), ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert (ws[size:] == 0xA5).all()
    want = ssd.linear_bwd(dy, x, w, ssd.unpack_rows(pre, ps), act="silu", want_dbias=True)
    assert torch.equal(dx, want["dx"]) and torch.equal(db, want["dbias"]) and (not want_dw or torch.equal(dw, want["dw"]))


@pytest.mark.parametrize("which", ["no x", "codes of x that are not read", "x in bf16"])
def test_what_a_call_allocates(which):
    from mamba_ssd_chunked_scan_gb300 import _lib as L
    x, w, dy, (pre, ps) = make(2, 8192, 256, 2560)
    args = dict(pre=pre, act="silu", pre_scales=ps)
    if which == "no x":
        args.update(x=None, want_dw=False)
    elif which == "x in bf16":
        args.update(x=x)
    else:
        args["x"], args["x_scales"] = ssd.pack_rows(x)
        args.update(want_dw=False)
    del x
    ssd.linear_bwd(dy, w=w, **args)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    got = ssd.linear_bwd(dy, w=w, **args)
    torch.cuda.synchronize()
    peak = torch.cuda.max_memory_allocated() - before
    outputs = sum(t.numel() * t.element_size() for t in got.values() if t is not None)
    # linear_bwd's workspace (dpre, and the parts of a product that is split along its contraction), and what the allocator rounds up
    plain = L.lib.ssd_linear_bwd_workspace_size(ctypes.byref(L.LinearParams(8192, 2560, 256, 2560, 1, 1))) + (1 << 20)
    assert peak <= outputs + plain, (peak, outputs, plain)


def test_codes_that_are_not_read_are_still_checked():
    x, w, dy, (pre, ps) = make(3, 16, 24, 48)
    xq, xs = ssd.pack_rows(x)
    full = ssd.linear_bwd(dy, xq, w, pre, act="silu", x_scales=xs, pre_scales=ps)
    wide = torch.zeros(16, 51, dtype=torch.uint8, device="cuda").view(E4)   # columns of a wider matrix, at an odd stride
    wide.view(torch.uint8)[:, :48] = xq.view(torch.uint8)
    got = ssd.linear_bwd(dy, wide[:, :48], w, pre, act="silu", x_scales=xs, pre_scales=ps, want_dw=False)
    assert got["dw"] is None and torch.equal(got["dx"], full["dx"])
    for bad in (dict(x=xq, x_scales=xs[:5]), dict(x=xq[:, :40], x_scales=xs), dict(x=xq, x_scales=xs.double()), dict(x=xq.t(), x_scales=xs)):
        with pytest.raises(ValueError):
            ssd.linear_bwd(dy, w=w, pre=pre, act="silu", pre_scales=ps, want_dw=False, **bad)
    with pytest.raises(TypeError):
        ssd.linear_bwd(dy, x, w, pre, act="silu", x_scales=xs, pre_scales=ps, want_dw=False)
