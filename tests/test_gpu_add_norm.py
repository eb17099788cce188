"""The residual RMS norm and its gradient on the GPU against the formula in 64 bits.

Bounds, derived from the kernels' arithmetic: a row's fp32 sum adds 16 products
per thread, 5 shuffles and at most 32 partials, so its relative error is under
54 * 2^-24 (all terms positive) and rstd's half of that; h, the product with
rstd and the one with the weight round once each.  FP = 64 * 2^-24 covers them.
A bf16 output (8 significant bits) rounds once more, by at most 2^-8 of its value; an e4m3 one by at
most 2^-4 of it, or half of the smallest step, 2^-10, near zero."""
import numpy as np
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FP = 64 * U
OUT = {torch.float32: U, torch.bfloat16: 2.0 ** -8 * 1.01}
BF, F4, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def make(rows, width, dtype, rtype, seed, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def t(kind, scale):
        # an odd offset into a larger buffer takes the base off 16-byte alignment
        flat = torch.empty(rows * width + offset, dtype=kind, device="cuda")
        flat[offset:] = torch.randn(rows * width, generator=g, device="cuda").mul_(scale).to(kind)
        return flat[offset:].view(rows, width)

    w = torch.randn(width, generator=g, device="cuda") * 0.3 + 1
    return t(dtype, 1.0), (None if rtype is None else t(rtype, 4.0)), w


def formula(x, res, w, eps):
    h = x.double() + (0 if res is None else res.double())
    rstd = 1 / torch.sqrt((h * h).mean(-1) + eps)
    return h, rstd, h * rstd[:, None] * w.double()


def close(got, want, bound, what):
    worst = ((got.double() - want).abs() / bound).max().item()
    assert np.isfinite(worst) and worst <= 1, (what, worst)


SHAPES = [
    (1, 1, 0), (5, 3, 0), (3, 24, 0), (7, 31, 0), (4, 512, 0), (9, 513, 0), (6, 520, 1), (37, 2560, 0), (130, 2561, 0),
    (2, 5120, 0), (3, 8191, 0), (2, 16384, 0), (2, 16384, 3),
]
TYPES = [(BF, None, BF), (BF, F4, BF), (BF, BF, E4), (BF, F4, E4), (F4, F4, F4), (F4, None, E4)]


@pytest.mark.parametrize("rows,width,offset", SHAPES)
@pytest.mark.parametrize("dtype,rtype,otype", TYPES)
def test_forward(rows, width, offset, dtype, rtype, otype):
    x, res, w = make(rows, width, dtype, rtype, rows * 7 + width, offset)
    got = ssd.add_norm(x, w, res, eps=1e-5, out_dtype=otype, return_rstd=True)
    h, rstd, out = formula(x, res, w, 1e-5)
    close(got["rstd"], rstd, FP * rstd, "rstd")
    if res is not None:
        close(got["residual"], h, OUT[rtype] * h.abs() + U * h.abs() + 1e-30, "residual")
    else:
        assert got["residual"] is None
    if otype is E4:
        scale = out.abs().amax(-1).clamp(min=1e-30) / 448
        close(got["scales"], scale, 2 * FP * scale, "scales")
        v = out / scale[:, None]
        close(got["out"].float(), v, (2.0 ** -4 + 4 * FP) * v.abs().clamp(min=2.0 ** -6), "e4m3")
        assert got["out"].float().abs().amax(-1).min() == 448   # the largest element takes the largest number
    else:
        assert got["scales"] is None
        close(got["out"], out, (OUT[otype] + FP) * out.abs() + 1e-30, "out")


@pytest.mark.parametrize("rows,width,offset", SHAPES + [(5000, 264, 0), (3001, 777, 0)])
@pytest.mark.parametrize("dtype,rtype", [(BF, BF), (BF, F4), (F4, F4)])
@pytest.mark.parametrize("with_res", [True, False])
def test_backward(rows, width, offset, dtype, rtype, with_res):
    dout, h, w = make(rows, width, dtype, rtype, rows + 3 * width, offset)
    dres = make(rows, width, dtype, rtype, rows + 5, offset)[1] if with_res else None
    rstd = (1 / torch.sqrt((h.double() ** 2).mean(-1) + 1e-5)).float()
    got = ssd.add_norm_bwd(dout, h, w, rstd, dres)
    r = rstd.double()[:, None]
    xh, p = h.double() * r, dout.double() * w.double()
    dot, dot_abs = (p * xh).mean(-1, keepdim=True), (p * xh).abs().mean(-1, keepdim=True)
    dh = r * (p - xh * dot) + (0 if dres is None else dres.double())
    slack = FP * (r * (p.abs() + 2 * xh.abs() * dot_abs) + dh.abs())
    close(got["dx"], dh, OUT[dtype] * dh.abs() + slack, "dx")
    close(got["dresidual"], dh, OUT[rtype] * dh.abs() + slack, "dresidual")
    # every share sums at most its rows one after another, then up to 32 warps of shares
    terms = dout.double() * xh
    close(got["dweight"], terms.sum(0), (rows + 64) * U * terms.abs().sum(0) + 1e-30, "dweight")


# rows of every shift against 16 bytes, several to a slot; the widest spans of each kernel shape; fewer columns than a vector
@pytest.mark.parametrize("rows,width", [(2500, 5), (1300, 9), (700, 1283), (1251, 1276), (500, 4001), (330, 5114), (320, 6001),
                                        (310, 8177), (310, 8186), (160, 16377), (155, 16378)])
@pytest.mark.parametrize("dtype,rtype", [(BF, BF), (BF, F4), (F4, F4)])
def test_backward_rows_off_16_bytes(rows, width, dtype, rtype):
    test_backward(rows, width, 0, dtype, rtype, True)
    test_backward(rows, width, 1, dtype, rtype, False)


@pytest.mark.parametrize("width", [1283, 4001, 333])
def test_backward_neighbouring_rows_stay_apart(width):
    """A row of NaNs or infinities reaches dweight, and no other row's gradient."""
    dout, h, w = make(912, width, BF, BF, width)
    rstd = (1 / torch.sqrt((h.double() ** 2).mean(-1) + 1e-5)).float()
    clean = ssd.add_norm_bwd(dout, h, w, rstd)["dx"]
    dout[5], h[8] = float("nan"), float("inf")
    got = ssd.add_norm_bwd(dout, h, w, rstd)["dx"]
    keep = torch.ones(912, dtype=torch.bool, device="cuda")
    keep[[5, 8]] = False
    assert torch.equal(got[keep], clean[keep]) and not got[~keep].isfinite().any()


def test_gradient_against_differences():
    x, res, w = make(6, 200, F4, F4, 11)
    g = torch.Generator(device="cuda").manual_seed(5)
    dout, dres, dirn = (torch.randn(6, 200, generator=g, device="cuda") for _ in range(3))
    f = ssd.add_norm(x, w, res, return_rstd=True)
    got = ssd.add_norm_bwd(dout, f["residual"], w, f["rstd"], dres)

    def value(step):
        h, _, out = formula(x.double() + step * dirn.double(), res, w, 1e-5)
        return (out * dout.double()).sum() + (h * dres.double()).sum()

    # central differences in 64 bits: their error is O(step^2), here under 1e-7 of the value
    slope = (value(1e-4) - value(-1e-4)) / 2e-4
    mine = (got["dx"].double() * dirn.double()).sum()
    assert abs(mine - slope) <= 1e-5 * (got["dx"].double() * dirn.double()).abs().sum()


def test_rows_that_hold_nothing_or_everything():
    w = torch.ones(300, device="cuda")
    x = torch.zeros(6, 300, device="cuda")
    x[1, 7] = float("inf")
    x[2, 9] = float("nan")
    x[3] = 1e-25          # squares underflow: only eps remains
    x[4] = 1e25           # squares overflow: rstd is zero
    x[5, 299] = -2.0
    for out_dtype in (F4, E4):
        got = ssd.add_norm(x, w, eps=1e-5, out_dtype=out_dtype)
        o = got["out"].float()
        assert (o[0] == 0).all() and o[2].isnan().all()
        assert o[1, 7].isnan()
        if out_dtype is E4:
            assert got["scales"][0] == np.float32(1e-30) / np.float32(448)
            assert got["scales"][1:3].isnan().all() and o[1].isnan().all()
            assert o[5, 299] == -448 and (o[3] == 448).all()
        else:
            assert (o[1, :7] == 0).all() and (o[4] == 0).all()
            assert torch.allclose(o[3], x[3] / 1e-5 ** 0.5, rtol=1e-5, atol=0)
    assert torch.isfinite(ssd.add_norm(x[:1], w, eps=1e-5)["out"]).all()


def test_no_rows():
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    got = ssd.add_norm(x, w, x, out_dtype=E4, return_rstd=True)
    assert got["out"].shape == (0, 64) and got["scales"].shape == (0,)
    back = ssd.add_norm_bwd(x, x, w, got["rstd"])
    assert back["dx"].shape == (0, 64) and (back["dweight"] == 0).all()


def test_leading_dimensions_stream_and_repeat():
    x, res, w = make(24, 136, BF, F4, 3)
    one = ssd.add_norm(x, w, res, return_rstd=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    two = ssd.add_norm(x.view(2, 3, 4, 136), w, res.view(2, 3, 4, 136), return_rstd=True, stream=s)
    s.synchronize()
    assert two["rstd"].shape == (2, 3, 4)
    assert torch.equal(one["out"], two["out"].view(24, 136)) and torch.equal(one["residual"], two["residual"].view(24, 136))
    dout = make(24, 136, BF, F4, 9)[0]
    a = ssd.add_norm_bwd(dout, res, w, one["rstd"], res)
    b = ssd.add_norm_bwd(dout, res, w, one["rstd"], res)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_in_place_through_the_c_entry():
    from mamba_ssd_chunked_scan_gb300 import _lib
    x, res, w = make(33, 264, BF, F4, 21)
    want = ssd.add_norm(x, w, res)
    st = torch.cuda.current_stream().cuda_stream
    rc = _lib.lib.ssd_add_norm(33, 264, 1, 0, 1, x.data_ptr(), res.data_ptr(), w.data_ptr(), 1e-5, x.data_ptr(), None,
                               res.data_ptr(), None, st)
    assert rc == 0
    assert torch.equal(x, want["out"]) and torch.equal(res, want["residual"])


def test_tensors_refused():
    x, res, w = make(4, 64, BF, F4, 1)
    for bad in (lambda: ssd.add_norm(x.half(), w), lambda: ssd.add_norm(x, w, out_dtype=F4),
                lambda: ssd.add_norm(x.float(), w, res.to(BF)), lambda: ssd.add_norm(x, w, res, residual_dtype=BF)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ssd.add_norm(x.cpu(), w), lambda: ssd.add_norm(x[:, ::2], w[:32]), lambda: ssd.add_norm(x, w[:32]),
                lambda: ssd.add_norm(x, w, res[:3]), lambda: ssd.add_norm(x, w.cpu()),
                lambda: ssd.add_norm_bwd(x, res, w, w[:3])):
        with pytest.raises(ValueError):
            bad()
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(ssd.SSDError):
            ssd.add_norm(x, w, eps=eps)
    wide = torch.zeros(1, 16385, device="cuda")
    with pytest.raises(ssd.SSDError):
        ssd.add_norm(wide, wide[0])
