"""The gate and norm after the scan with its 8-bit checkpoint, and its gradient, against the formulas in 64 bits.

A gradient's bound is FP times the sizes of the terms that it sums (norms_helpers) and half a step of its type."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
from norms_helpers import BF, F4, FP, HALF, U, close, gate, mean, norm_bwd, rows_by_table, same_codes, wide

pytestmark = pytest.mark.gpu

EPS = 1e-5


def columns(v, extra, offset=0):
    """v as columns of a matrix `extra` wider, `offset` elements into its buffer."""
    rows, width = v.shape
    flat = torch.zeros(rows * (width + extra) + offset, dtype=v.dtype, device="cuda")
    out = flat[offset:].view(rows, width + extra)[:, :width]
    out.copy_(v)
    return out


def make(rows, width, dtype, seed, extra=0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda scale: torch.randn(rows, width, generator=g, device="cuda") * scale
    y, z, d = r(0.7), r(2.0).clamp(-15, 15), r(1.0)
    y[rows // 2] = 0   # a row that holds nothing
    w = torch.randn(width, generator=g, device="cuda") * 0.3 + 1
    c = lambda v, e: columns(v.to(dtype), e, offset)
    return c(y, 0), c(z, extra), c(d, 0), w


SHAPES = [(1, 1, 1, 0, 0), (5, 3, 1, 0, 0), (3, 24, 3, 0, 0), (7, 31, 1, 5, 0), (4, 512, 1, 16, 0), (9, 513, 1, 0, 0), (6, 520, 1, 8, 1),
          (37, 2560, 1, 80, 0), (130, 2561, 1, 0, 0), (12, 5120, 80, 5456, 0), (3, 8191, 1, 0, 0), (2, 8192, 1, 0, 3), (700, 264, 1, 0, 0),
          (300, 1536, 3, 0, 0), (2500, 5, 1, 0, 0), (1300, 72, 8, 0, 0), (333, 1283, 1, 0, 0), (2, 16384, 2, 8, 0), (1, 4096, 4096, 0, 0)]


@pytest.mark.parametrize("rows,width,groups,extra,offset", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F4])
def test_forward_and_what_it_keeps(rows, width, groups, extra, offset, dtype):
    y, z, _, w = make(rows, width, dtype, rows + width, extra, offset)
    out, kept = ssd.gate_norm(y, z, w, width // groups, EPS, pack=True)
    u = y.double() * gate(z.double())[0]
    want = u * torch.rsqrt(mean(u * u, groups) + EPS) * w.double()
    close(out, want, (HALF[dtype] + FP) * want.abs() + 1e-30, "out")
    for name, t in (("y", y), ("z", z)):
        codes, scales = rows_by_table(t, groups)
        assert kept[name + "_scales"].shape == (rows, groups)
        assert torch.equal(kept[name + "_scales"].cpu(), scales) and same_codes(kept[name], codes), name


def check(got, dout, y, z, w, groups, dtype, want_out):
    yd, zd, do = y, z, dout.double()
    a, slope, slope_size = gate(zd)
    u = yd * a
    du, size, n, r = norm_bwd(do, u, w.double(), EPS, groups)
    close(got["dy"], du * a, HALF[dtype] * (du * a).abs() + FP * size * a.abs() + 1e-30, "dy")
    dz = du * yd * slope
    close(got["dz"], dz, HALF[dtype] * dz.abs() + 2 * FP * size * yd.abs() * slope_size + 1e-30, "dz")
    terms = do * n
    close(got["dweight"], terms.sum(0), ((dout.shape[0] + 64) * U + FP) * terms.abs().sum(0) + 1e-30, "dweight")
    if want_out:
        out = n * w.double()
        close(got["out"], out, (HALF[dtype] + FP) * out.abs() + 1e-30, "out")
    else:
        assert got["out"] is None


@pytest.mark.parametrize("rows,width,groups,extra,offset", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F4])
def test_gradient(rows, width, groups, extra, offset, dtype):
    y, z, d, w = make(rows, width, dtype, rows + 3 * width, extra, offset)
    whole = torch.full((rows, width + extra), 7.0, dtype=dtype, device="cuda")
    got = ssd.gate_norm_bwd(d, y, z, w, width // groups, EPS, dz=whole[:, :width], want_out=bool(rows % 2))
    check(got, d, y.double(), z.double(), w, groups, dtype, bool(rows % 2))
    assert (whole[:, width:] == 7).all()   # the neighbouring columns are left alone
    assert got["dz"].data_ptr() == whole.data_ptr()


@pytest.mark.parametrize("rows,width,groups,extra,offset", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F4])
@pytest.mark.parametrize("which", ["yz", "y", "z"])
def test_gradient_from_the_checkpoint(rows, width, groups, extra, offset, dtype, which):
    y, z, d, w = make(rows, width, dtype, rows + 5 * width, extra, offset)
    kept = ssd.gate_norm(y, z, w, width // groups, EPS, pack=True)[1]
    args = {"y": y, "z": z}
    for name in which:
        args[name], args[name + "_scales"] = kept[name], kept[name + "_scales"]
    got = ssd.gate_norm_bwd(d, weight=w, group_size=width // groups, eps=EPS, want_out=True, **args)
    check(got, d, wide(args["y"], args.get("y_scales")), wide(args["z"], args.get("z_scales")), w, groups, dtype, True)


def test_gradient_against_differences():
    y, z, d, w = make(6, 200, F4, 11)
    got = ssd.gate_norm_bwd(d, y, z, w, 100, EPS)
    g = torch.Generator(device="cuda").manual_seed(5)
    ty, tz = (torch.randn(6, 200, generator=g, device="cuda").double() for _ in range(2))
    tw = torch.randn(200, generator=g, device="cuda").double()

    def value(step):
        zs = z.double() + step * tz
        u = (y.double() + step * ty) * zs / (1 + torch.exp(-zs))
        return (u * torch.rsqrt(mean(u * u, 2) + EPS) * (w.double() + step * tw) * d.double()).sum()

    # central differences in 64 bits: their error is O(step^2) of the third derivative
    slope = (value(1e-5) - value(-1e-5)) / 2e-5
    terms = torch.cat([(got["dy"].double() * ty).flatten(), (got["dz"].double() * tz).flatten(), got["dweight"].double() * tw])
    assert abs(terms.sum() - slope) <= 1e-5 * terms.abs().sum()


@pytest.mark.parametrize("width", [1283, 2560, 333, 64])
@pytest.mark.parametrize("packed", [False, True])
def test_rows_stay_apart(width, packed):
    """Rows of NaNs or infinities reach dweight, and no other row."""
    y, z, d, w = make(912, width, BF, width)
    call = lambda: ssd.gate_norm_bwd(d, weight=w, group_size=width, want_out=True,
                                     **(ssd.gate_norm(y, z, w, width, pack=True)[1] if packed else dict(y=y, z=z)))
    clean = call()
    d[5], y[8], z[11, 3] = float("nan"), float("inf"), float("nan")
    got = call()
    keep = torch.ones(912, dtype=torch.bool, device="cuda")
    keep[[5, 8, 11]] = False
    for name in ("dy", "dz", "out"):
        assert torch.equal(got[name][keep], clean[name][keep]), name
        assert name == "out" or not got[name][5].isfinite().any()
    assert got["dweight"].isnan().all()


def test_extreme_gates():
    """Gates closed and wide open: silu and its slope at their limits."""
    z = torch.tensor([-1e4, -200.0, -88.0, -30.0, 0.0, 30.0, 88.0, 200.0, 1e4, 1.0], device="cuda").repeat(4, 1)
    y = torch.ones_like(z)
    d = torch.randn(4, 10, device="cuda")
    w = torch.ones(10, device="cuda")
    for dtype in (F4, BF):
        got = ssd.gate_norm_bwd(d.to(dtype), y.to(dtype), z.to(dtype), w, 10, want_out=True)
        assert all(t.isfinite().all() for t in got.values())
        assert (got["dy"][:, :2] == 0).all() and (got["dz"][:, :2] == 0).all() and (got["out"][:, :2].abs() == 0).all()


def test_nothing_and_dimensions():
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    out, kept = ssd.gate_norm(x, x, w, 32, pack=True)
    assert out.shape == (0, 64) and kept["z_scales"].shape == (0, 2)
    got = ssd.gate_norm_bwd(x, weight=w, group_size=32, want_out=True, **kept)
    assert got["dy"].shape == (0, 64) and (got["dweight"] == 0).all()
    y, z, d, w = make(24, 136, BF, 3)
    one = ssd.gate_norm_bwd(d, y, z, w, 136)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    two = ssd.gate_norm_bwd(d.view(2, 3, 4, 136), y.view(2, 3, 4, 136), z.view(2, 3, 4, 136), w, 136, stream=s)
    s.synchronize()
    assert two["dy"].shape == (2, 3, 4, 136)
    for k in ("dy", "dz", "dweight"):
        assert torch.equal(one[k].flatten(), two[k].flatten())


def test_refusals():
    y, z, d, w = make(4, 64, BF, 1)
    kept = ssd.gate_norm(y, z, w, 32, pack=True)[1]
    bwd = lambda **kw: ssd.gate_norm_bwd(**{**dict(dout=d, y=y, z=z, weight=w, group_size=32), **kw})
    for bad in (lambda: ssd.gate_norm(y.half(), z, w, 64, pack=True), lambda: bwd(dout=d.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ssd.gate_norm(y, z, w, 64, out=y, pack=True), lambda: ssd.gate_norm(y, z, w, 48, pack=True), lambda: bwd(group_size=0),
                lambda: bwd(y=kept["y"]), lambda: bwd(y_scales=kept["y_scales"]), lambda: bwd(z=z[:3]), lambda: bwd(z=z.t()), lambda: bwd(weight=w[:5]),
                lambda: bwd(z=kept["z"], z_scales=kept["z_scales"][:, :1]), lambda: bwd(dz=torch.empty(4, 64, device="cuda")),
                lambda: bwd(y=torch.zeros(4, 128, dtype=BF, device="cuda")[:, :64]), lambda: bwd(dout=d.cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: bwd(eps=-1.0), lambda: bwd(eps=float("nan")), lambda: bwd(dz=z), lambda: bwd(dz=d)):
        with pytest.raises(ssd.SSDError):
            bad()
    big = torch.zeros(1, 8193, device="cuda")
    with pytest.raises(ssd.SSDError):
        ssd.gate_norm_bwd(big, big, big, big[0], 8193)
