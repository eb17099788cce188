"""A projection's gradients from 8-bit rows against the formula in 64 bits.

x in 8 bits stands for a bf16 number where its scale is a power of two, so the products are those of linear_bwd; dpre is
formed from the activation's argument in fp32 and rounded to bf16 as the products' operand."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
from norms_helpers import BF, E4, U, close, wide

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8 * 1.01


def make(m, n, k, seed, act, scales, extra=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    if scales == "packed":
        x, xs = ssd.pack_rows(r(m, k))
    else:
        q = ssd.add_norm(r(m, k), torch.rand(k, generator=g, device="cuda") + 0.5, out_dtype=E4)
        x, xs = q["out"], q["scales"]
    if extra:
        full = torch.zeros(m, k + extra, dtype=torch.uint8, device="cuda").view(E4)
        full.view(torch.uint8)[:, :k] = x.view(torch.uint8)
        x = full[:, :k]
    pre = ps = None
    if act != "none":
        pre, ps = ssd.pack_rows(r(m, n) * 2)
    return x, xs, (r(n, k) / k ** 0.5).to(BF), r(m, n).to(BF), pre, ps


def slope(v, act):
    v = v.detach().requires_grad_(True)
    y = {"none": lambda u: u, "silu": torch.nn.functional.silu, "gelu": lambda u: torch.nn.functional.gelu(u, approximate="tanh")}[act](v)
    return torch.autograd.grad(y.sum(), v)[0]


@pytest.mark.parametrize("m,n,k,extra", [(1, 8, 16, 0), (7, 33, 24, 3), (64, 200, 64, 0), (129, 96, 136, 16), (300, 513, 256, 0), (1000, 640, 1288, 1)])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("scales", ["packed", "amax"])
def test_gradients(m, n, k, extra, act, scales):
    x, xs, w, dy, pre, ps = make(m, n, k, m + n, act, scales, extra)
    got = ssd.linear_bwd(dy, x, w, pre, act=act, x_scales=xs, pre_scales=ps, want_dbias=True, check_status=True)
    d = dy.double()
    # the slopes' errors (a few 2^-22 of terms below 2) and dpre's rounding as an operand; scales that are no powers of two are in it
    # where it is an array of its own, otherwise x is rounded
    off, own = torch.zeros_like(d), act != "none" or n % 8 != 0
    if act != "none":
        d = d * slope(wide(pre, ps), act)
        off = 64 * U * dy.double().abs() + HALF * d.abs()
    elif own and scales != "packed":
        off = HALF * d.abs()
    xd, wd = wide(x, xs), w.double()
    off_x = 0 if scales == "packed" or own else HALF * xd.abs()
    sums = (2 * max(m, n, k) + 64) * U
    dx, dw = d @ wd, d.t() @ xd
    close(got["dx"], dx, HALF * dx.abs() + off @ wd.abs() + sums * (d.abs() @ wd.abs()) + 1e-30, "dx")
    size = d.abs().t() @ xd.abs()
    close(got["dw"], dw, HALF * dw.abs() + off.t() @ xd.abs() + (0 if isinstance(off_x, int) else d.abs().t() @ off_x) + sums * size + 1e-30, "dw")
    close(got["dbias"], d.sum(0), (64 * U * dy.double().abs()).sum(0) + sums * d.abs().sum(0) + 1e-30, "dbias")


@pytest.mark.parametrize("m,n,k", [(64, 200, 64), (300, 513, 256), (777, 1000, 328)])
def test_the_same_bits_as_from_bf16(m, n, k):
    """pack_rows' rows lose nothing on the way to the products."""
    x, xs, w, dy, pre, ps = make(m, n, k, 5, "silu", "packed")
    full = ssd.unpack_rows(x, xs)
    a = ssd.linear_bwd(dy, x, w, x_scales=xs)
    b = ssd.linear_bwd(dy, full, w)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"])
    # pre alone in 8 bits, and x alone
    pf = ssd.unpack_rows(pre, ps)
    want = ssd.linear_bwd(dy, full, w, pf, act="silu", want_dbias=True)
    for args in (dict(x=full, pre=pre, pre_scales=ps), dict(x=x, x_scales=xs, pre=pf), dict(x=x, x_scales=xs, pre=pre, pre_scales=ps)):
        got = ssd.linear_bwd(dy, w=w, act="silu", want_dbias=True, **args)
        for name in want:
            assert torch.equal(got[name], want[name]), name


def test_only_what_is_wanted_and_nothing():
    x, xs, w, dy, pre, ps = make(100, 72, 48, 3, "gelu", "packed")
    every = ssd.linear_bwd(dy, x, w, pre, act="gelu", x_scales=xs, pre_scales=ps, want_dbias=True)
    for name in ("dx", "dw", "dbias"):
        wants = {"want_" + k: k == name for k in ("dx", "dw", "dbias")}
        got = ssd.linear_bwd(dy, x, w, pre, act="gelu", x_scales=xs, pre_scales=ps, **wants)
        assert torch.equal(got[name], every[name]) and sum(v is not None for v in got.values()) == 1
    got = ssd.linear_bwd(dy[:0], x[:0], w, pre[:0], act="gelu", x_scales=xs[:0], pre_scales=ps[:0], want_dbias=True)
    assert got["dx"].shape == (0, 48) and (got["dw"] == 0).all() and (got["dbias"] == 0).all()
    nan = x.view(torch.uint8).clone()
    nan[5, 3] = 127   # e4m3's NaN reaches its column of dw, and nothing else
    got = ssd.linear_bwd(dy, nan.view(E4), w, pre, act="gelu", x_scales=xs, pre_scales=ps)
    assert got["dw"][:, 3].isnan().all() and torch.equal(got["dx"], every["dx"])
    keep = torch.arange(48, device="cuda") != 3
    assert torch.equal(got["dw"][:, keep], every["dw"][:, keep])


def test_refusals():
    x, xs, w, dy, pre, ps = make(16, 24, 48, 3, "silu", "packed")
    bwd = lambda **kw: ssd.linear_bwd(**{**dict(dy=dy, x=x, w=w, pre=pre, act="silu", x_scales=xs, pre_scales=ps), **kw})
    for bad in (lambda: bwd(x=x.float().to(BF)), lambda: bwd(x_scales=None)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for bad in (lambda: bwd(x_scales=xs[:5]), lambda: bwd(pre_scales=None), lambda: bwd(pre_scales=ps.double()), lambda: bwd(act="none"),
                lambda: bwd(act="none", pre=None), lambda: bwd(w=w.float()), lambda: bwd(w=w[:, :40]), lambda: bwd(act="relu")):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ssd.SSDError):   # k is a multiple of 8
        ssd.linear_bwd(dy, x[:, :44].contiguous(), w[:, :44].contiguous(), x_scales=xs)


def test_without_the_operand():
    """dx and dbias need no x: the same bits without it, and from bf16 pre as from 8-bit rows' values."""
    g = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    x, w, dy = r(2, 77, 64), r(40, 64), r(2, 77, 40)
    codes, scales = ssd.pack_rows(r(2, 77, 40))
    for pre in (ssd.unpack_rows(codes, scales), None):
        act = "none" if pre is None else "silu"
        want = ssd.linear_bwd(dy, x, w, pre, act=act, want_dbias=True)
        got = ssd.linear_bwd(dy, None, w, pre, act=act, want_dw=False, want_dbias=True)
        assert got["dw"] is None and torch.equal(got["dx"], want["dx"]) and torch.equal(got["dbias"], want["dbias"])
    want = ssd.linear_bwd(dy, x, w, ssd.unpack_rows(codes, scales), act="silu", want_dw=False)
    got = ssd.linear_bwd(dy, None, w, codes, act="silu", pre_scales=scales, want_dw=False)
    assert torch.equal(got["dx"], want["dx"])
    assert torch.equal(ssd.linear_bwd(dy, None, w, want_dw=False, want_dx=False, want_dbias=True)["dbias"],
                       ssd.linear_bwd(dy, x, w, want_dw=False, want_dx=False, want_dbias=True)["dbias"])
