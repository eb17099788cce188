"""The projection with its epilogue, and its gradients, on the GPU against the formula in 64 bits.

Bounds.  With U = 2^-24 the products of bf16 (and of e4m3) numbers are exact in fp32 and 16 of them at least
are added to a running fp32 sum at a time, so a sum over k is within (k / 16 + 32) 2 U of the sum of the
magnitudes.  Both activations change by at most 1.13 times their argument's change.  y rounds to
bf16 once (2^-8 of its value).  The gradients' operand dpre is rounded to bf16 where there is an
activation, 2^-8 of each term of the sums.  Products of small integers have to be exact."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B8 = 2.0 ** -8 * 1.01
BF, F4, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def close(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    worst = ((got.double() - want).abs() / (bound + 1e-30)).max().item()
    assert worst <= 1, (what, worst)


def activation(v, act):
    if act == "silu":
        return torch.nn.functional.silu(v)
    return torch.nn.functional.gelu(v, approximate="tanh") if act == "gelu" else v


SHAPES = [   # rows, columns, contraction
    (1, 1, 16), (1, 33, 64), (2, 1000, 16), (8, 640, 2560), (15, 130, 80), (16, 128, 128), (17, 257, 144), (33, 96, 512),
    (64, 2000, 272), (65, 64, 64), (100, 1, 96), (127, 129, 48), (128, 128, 256), (129, 255, 1040), (300, 520, 2048),
    (1000, 72, 5120), (2000, 3000, 144), (4099, 264, 640),
]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("kind", [BF, E4])
def test_whole_numbers_are_exact(m, n, k, kind):
    g = gen(m + n + k)
    # entries -1, 0, 1, few of w's not 0: sums stay under 256, where bf16 holds every whole number
    x = torch.randint(-1, 2, (m, k), generator=g, device="cuda").float()
    w = torch.randint(-1, 2, (n, k), generator=g, device="cuda").float() * (torch.rand(n, k, generator=g, device="cuda") < 60 / k)
    want = x.double() @ w.double().t()
    assert want.abs().max() <= 256
    s = (None, None) if kind is BF else (torch.full((m,), 0.5, device="cuda"), torch.full((n,), 2.0, device="cuda"))
    y = ssd.linear(x.to(kind), w.to(kind), x_scales=s[0], w_scales=s[1], check_status=True)
    assert torch.equal(y.double(), want)


def rows_e4m3(v):
    s = v.abs().amax(-1) / 448
    return (v / s[:, None]).clamp(-448, 448).to(E4), s


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("act,bias,res,pre", [("none", False, False, False), ("silu", True, True, True), ("gelu", True, False, False),
                                              ("none", False, True, True)])
def test_forward(m, n, k, kind, act, bias, res, pre):
    g = gen(3 * m + n + k)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, w = r(m, k), r(n, k) / k ** 0.5
    xs = ws = None
    if kind is E4:
        (x, xs), (w, ws) = rows_e4m3(x), rows_e4m3(w)
    else:
        x, w = x.to(BF), w.to(BF)
    b = r(n) if bias else None
    q = (r(m, n) * 3).to(BF) if res else None
    got = ssd.linear(x, w, b, q, act=act, x_scales=xs, w_scales=ws, return_pre=pre, check_status=True)
    y, p = got if pre else (got, None)
    xd, wd = x.double(), w.double()
    if xs is not None:
        xd, wd = xd * xs.double()[:, None], wd * ws.double()[:, None]
    v = xd @ wd.t()
    slack = (k / 16 + 40) * 2 * U * (xd.abs() @ wd.abs().t())
    if b is not None:
        v = v + b.double()
        slack = slack + 2 * U * (v.abs() + b.double().abs())
    if pre:
        close(p, v, B8 * v.abs() + slack, "pre")
    want = activation(v, act)
    slack = 1.13 * slack + 64 * U * (v.abs() + want.abs())
    if q is not None:
        want = want + q.double()
    close(y, want, B8 * want.abs() + slack + U * want.abs(), "y")


GRAD = [(16, 64, 64), (1, 40, 24), (50, 33, 128), (130, 129, 136), (300, 1, 64), (257, 520, 200), (1000, 264, 72), (3000, 64, 32),
        (2100, 1500, 1288), (2600, 3300, 1288)]


@pytest.mark.parametrize("m,n,k", GRAD)
def test_whole_number_gradients_are_exact(m, n, k):
    g = gen(m + n)
    pick = lambda *s, share: torch.randint(-1, 2, s, generator=g, device="cuda").float() * (torch.rand(*s, generator=g, device="cuda") < share)
    dy, x, w = pick(m, n, share=min(1, 60 / max(m, n))), pick(m, k, share=1), pick(n, k, share=1)
    got = ssd.linear_bwd(dy.to(BF), x.to(BF), w.to(BF), want_dbias=True, check_status=True)
    for name, want in (("dx", dy.double() @ w.double()), ("dw", dy.double().t() @ x.double()), ("dbias", dy.double().sum(0))):
        assert want.abs().max() <= 256
        assert torch.equal(got[name].double(), want), name


@pytest.mark.parametrize("m,n,k", GRAD)
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_gradients(m, n, k, act):
    g = gen(m + 2 * n + k)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, w, dy = r(m, k).to(BF), (r(n, k) / k ** 0.5).to(BF), r(m, n).to(BF)
    pre = None if act == "none" else (r(m, n) * 2).to(BF)
    got = ssd.linear_bwd(dy, x, w, pre, act=act, want_dbias=True, check_status=True)
    d = dy.double()
    if pre is not None:
        v = pre.double().requires_grad_(True)
        d = torch.autograd.grad(activation(v, act), v, d)[0]
        err = B8 * d.abs() + 64 * U * dy.double().abs() * 1.2
    else:
        err = torch.zeros_like(d)
    xd, wd = x.double(), w.double()
    dx, dw = d @ wd, d.t() @ xd
    close(got["dx"], dx, B8 * dx.abs() + 1.01 * (err @ wd.abs()) + (n / 16 + 40) * 2 * U * (d.abs() @ wd.abs()), "dx")
    close(got["dw"], dw, B8 * dw.abs() + 1.01 * (err.t() @ xd.abs()) + (m / 16 + 40) * 2 * U * (d.abs().t() @ xd.abs()), "dw")
    close(got["dbias"], d.sum(0), (m + 64) * U * d.abs().sum(0) + 64 * U * 1.2 * dy.double().abs().sum(0), "dbias")


def test_gradient_against_differences():
    g = gen(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    x, w, dy, b = r(20, 64), r(48, 64), r(20, 48), torch.randn(48, device="cuda", generator=g)
    y, pre = ssd.linear(x, w, b, act="gelu", return_pre=True)
    got = ssd.linear_bwd(dy, x, w, pre, act="gelu", want_dbias=True)

    def value(xx, ww, bb):
        return (activation(xx @ ww.t() + bb, "gelu") * dy.double()).sum()

    for name, t, d in (("dx", 0, r(20, 64)), ("dw", 1, r(48, 64)), ("dbias", 2, torch.randn(48, device="cuda", generator=g))):
        at = [x.double(), w.double(), b.double()]
        up, down = list(at), list(at)
        up[t], down[t] = at[t] + 1e-5 * d.double(), at[t] - 1e-5 * d.double()
        slope = (value(*up) - value(*down)) / 2e-5
        terms = got[name].double() * d.double()
        # pre and dpre are rounded to bf16: 2^-8 each, of pre's value (up to about 40 here) on the slope's argument
        assert abs(terms.sum() - slope) <= 0.02 * terms.abs().sum(), name


def test_rows_of_a_wider_matrix_and_leading_dimensions():
    g = gen(2)
    wide = torch.randn(3, 50, 400, generator=g, device="cuda").to(BF)
    w = torch.randn(72, 128, generator=g, device="cuda").to(BF)
    x = wide[..., 64:192]
    y = ssd.linear(x, w)
    assert y.shape == (3, 50, 72) and torch.equal(y, ssd.linear(x.contiguous(), w))
    dy = torch.randn(3, 50, 72, generator=g, device="cuda").to(BF)
    a, b = ssd.linear_bwd(dy, x, w), ssd.linear_bwd(dy, x.contiguous(), w)
    assert a["dx"].shape == x.shape and torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"])
    one = ssd.linear(x[0, 0], w)
    assert one.shape == (72,)


def test_infinities_and_nan_stay_in_their_rows():
    x = torch.zeros(70, 64, device="cuda", dtype=BF)
    w = torch.ones(40, 64, device="cuda", dtype=BF)
    x[3, 5], x[66, 9] = float("nan"), float("inf")
    x[4] = 1
    y = ssd.linear(x, w)
    assert y[3].isnan().all() and (y[66] == float("inf")).all() and (y[4] == 64).all()
    rest = torch.ones(70, dtype=torch.bool)
    rest[[3, 4, 66]] = False
    assert (y[rest.cuda()] == 0).all()


def test_in_place_residual_stream_and_repeat():
    from mamba_ssd_chunked_scan_gb300 import _lib
    import ctypes
    g = gen(7)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    for m in (9, 200):
        x, w, res = r(m, 256), r(512, 256), r(m, 512)
        want = ssd.linear(x, w, None, res)
        assert all(torch.equal(ssd.linear(x, w, None, res), want) for _ in range(3))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        other = ssd.linear(x, w, None, res, stream=s)
        s.synchronize()
        assert torch.equal(other, want)
        p = _lib.LinearParams(m, 256, 512, 256, 1, 0)
        ws = torch.empty(_lib.lib.ssd_linear_workspace_size(p), dtype=torch.uint8, device="cuda")
        rc = _lib.lib.ssd_linear(ctypes.byref(p), x.data_ptr(), w.data_ptr(), None, None, None, res.data_ptr(), res.data_ptr(), None,
                                 ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and torch.equal(res, want)


def test_outputs_off_16_byte_alignment():
    from mamba_ssd_chunked_scan_gb300 import _lib
    import ctypes
    g = gen(17)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    for m in (9, 200):
        x, w, res = r(m, 64), r(72, 64), r(m, 72)
        want = ssd.linear(x, w, None, res)
        flat = torch.zeros(m * 72 + 1, dtype=BF, device="cuda")
        p = _lib.LinearParams(m, 64, 72, 64, 1, 0)
        ws = torch.empty(_lib.lib.ssd_linear_workspace_size(p), dtype=torch.uint8, device="cuda")
        rc = _lib.lib.ssd_linear(ctypes.byref(p), x.data_ptr(), w.data_ptr(), None, None, None, res.data_ptr(), flat.data_ptr() + 2, None,
                                 ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and torch.equal(flat[1:].view(m, 72), want) and flat[0] == 0


def test_no_rows():
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(32, 64, dtype=BF, device="cuda")
    assert ssd.linear(x, w).shape == (0, 32)
    got = ssd.linear_bwd(torch.empty(0, 32, dtype=BF, device="cuda"), x, w, want_dbias=True)
    assert got["dx"].shape == (0, 64) and (got["dw"] == 0).all() and (got["dbias"] == 0).all()


def test_norm_rows_feed_the_product():
    g = gen(5)
    x, res = torch.randn(40, 256, generator=g, device="cuda").to(BF), torch.randn(40, 256, generator=g, device="cuda")
    weight, w = torch.rand(256, generator=g, device="cuda") + 0.5, torch.randn(96, 256, generator=g, device="cuda") / 16
    n = ssd.add_norm(x, weight, res, out_dtype=E4)
    wq, ws = rows_e4m3(w)
    y = ssd.linear(n["out"], wq, x_scales=n["scales"], w_scales=ws)
    full = ssd.add_norm(x, weight, res)["out"].double() @ w.double().t()
    # each operand is within 2^-4 of its value: the sum within an eighth of its terms' magnitudes, about
    # 1/8 / sqrt(256) of them at random; a quarter of the result's scale is far outside both
    assert ((y.double() - full).abs().max() / full.abs().max()) < 0.25
    want = (n["out"].double() * n["scales"].double()[:, None]) @ (wq.double() * ws.double()[:, None]).t()
    close(y, want, B8 * want.abs() + 1e-4, "y")


def test_tensors_refused():
    x, w = torch.zeros(4, 64, dtype=BF, device="cuda"), torch.zeros(32, 64, dtype=BF, device="cuda")
    s = torch.ones(4, device="cuda")
    for bad in (lambda: ssd.linear(x.float(), w.float()), lambda: ssd.linear_bwd(x, x.to(E4), w.to(E4))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ssd.linear(x, w[:, :32]), lambda: ssd.linear(x, w.float()), lambda: ssd.linear(x, w, act="tanh"),
                lambda: ssd.linear(x.cpu(), w), lambda: ssd.linear(x, w, s), lambda: ssd.linear(x, w, None, x),
                lambda: ssd.linear(x, w, x_scales=s), lambda: ssd.linear(x.to(E4), w.to(E4), x_scales=s),
                lambda: ssd.linear(x.to(E4), w.to(E4), x_scales=s, w_scales=s), lambda: ssd.linear(x.t(), w[:, :4]),
                lambda: ssd.linear_bwd(x, x, w), lambda: ssd.linear_bwd(torch.zeros(4, 32, dtype=BF, device="cuda"), x, w, act="silu"),
                lambda: ssd.linear(x, w.t().contiguous().t())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ssd.linear(x[:, :12].contiguous(), w[:, :12].contiguous()), lambda: ssd.linear(x.view(-1)[1:193].view(3, 64), w)):
        with pytest.raises(ssd.SSDError):
            bad()
