"""The norm after a block (gate, residual scale, the next block's norm) and its gradient against the formulas in 64 bits.

Bounds: FP times the sizes of the terms (norms_helpers), carried through the second norm, and half a step of the
output's type."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
from norms_helpers import BF, E4, F4, FP, HALF, U, close, gate, mean, norm_bwd, rows_by_table, same_codes, wide
from test_gpu_gate_norm_bwd import columns

pytestmark = pytest.mark.gpu

EPS, SCALE = 1e-5, 0.22
SHAPES = [(1, 1, 0, 0), (5, 3, 0, 0), (3, 24, 8, 0), (7, 31, 5, 0), (4, 512, 0, 0), (9, 513, 0, 0), (6, 520, 8, 1), (37, 2560, 80, 0), (130, 2561, 0, 0),
          (2, 5120, 0, 0), (3, 8191, 0, 0), (2, 8192, 16, 0), (700, 264, 0, 0), (500, 1533, 0, 0), (8, 2560, 0, 0), (1300, 9, 0, 0), (310, 4104, 0, 0)]
TYPES = [(BF, F4), (BF, BF), (F4, F4)]


def make(rows, width, dtype, rtype, seed, extra=0, offset=0, gated=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda scale: torch.randn(rows, width, generator=g, device="cuda") * scale
    c = lambda v, kind, e=0: columns(v.to(kind), e, offset)
    x = r(2.0)
    x[rows // 2] = 0
    t = dict(x=c(x, dtype), res=c(r(3.0), rtype), gate=c(r(2.0).clamp(-15, 15), dtype, extra) if gated else None, dout=c(r(1.0), dtype), dres=c(r(1.0), rtype))
    t["w"], t["w2"] = (torch.randn(width, generator=g, device="cuda") * 0.3 + 1 for _ in range(2))
    return t


def formula(t):
    u = t["x"].double() * (1 if t["gate"] is None else gate(t["gate"].double())[0])
    n = SCALE * u * torch.rsqrt(mean(u * u) + EPS) * t["w"].double()
    h = t["res"].double() + n
    r2 = torch.rsqrt(mean(h * h) + EPS)
    return n, h, r2, h * r2 * t["w2"].double()


@pytest.mark.parametrize("rows,width,extra,offset", SHAPES)
@pytest.mark.parametrize("dtype,rtype", TYPES)
@pytest.mark.parametrize("gated,out_dtype,pack", [(True, None, True), (False, E4, False), (True, E4, True), (False, None, True)])
def test_forward(rows, width, extra, offset, dtype, rtype, gated, out_dtype, pack):
    t = make(rows, width, dtype, rtype, rows + width, extra, offset, gated)
    got = ssd.block_norm(t["x"], t["w"], t["res"], t["gate"], t["w2"], scale=SCALE, eps=EPS, out_dtype=out_dtype, pack=pack)
    n, h, r2, out = formula(t)
    off_h = FP * n.abs() + 2 * U * h.abs()
    close(got["residual"], h, HALF[rtype] * h.abs() + off_h + 1e-30, "residual")
    # h's error reaches out by itself and through its row's norm
    off = FP * out.abs() + r2 * t["w2"].double().abs() * off_h + out.abs() * r2 * r2 * mean(h.abs() * off_h)
    if out_dtype is E4:
        # half a step of e4m3: 2^-4 of the number, or of the smallest normal one, at a scale of the smallest power of two that holds it
        s = got["scales"].double()[:, None]
        top = out.abs().amax(1, keepdim=True)
        tiny = 2.0 ** -108
        assert ((448 * s >= top * (1 - 4 * FP)) & ((224 * s < top * (1 + 4 * FP)) | (s == tiny))).all()
        assert torch.equal(torch.frexp(got["scales"])[0], torch.full_like(got["scales"], 0.5))
        close(wide(got["out"], got["scales"]), out, 2.0 ** -4 * out.abs().clamp(min=0) + 2.0 ** -10 * s + 2 * off, "e4m3")
    else:
        assert got["scales"] is None
        close(got["out"], out, HALF[dtype] * out.abs() + off + 1e-30, "out")
    for name in ("x", "gate"):
        if pack and t[name] is not None:
            codes, scales = rows_by_table(t[name])
            assert torch.equal(got[name + "_scales"].cpu(), scales[:, 0]) and same_codes(got[name], codes), name
        else:
            assert got[name] is None and got[name + "_scales"] is None
    one = ssd.block_norm(t["x"], t["w"], t["res"], t["gate"], scale=SCALE, eps=EPS)
    assert one["out"] is None and torch.equal(one["residual"], got["residual"])


def check(got, t, x, z, h, dtype, rtype, next_norm):
    d = t["dres"].double()
    off_dh = 2 * U * d.abs()
    if next_norm:
        dh2, size2, n2, r2 = norm_bwd(t["dout"].double(), h, t["w2"].double(), EPS)
        dh = d + dh2
        off_dh = off_dh + FP * size2 + 2 * U * dh.abs()
        terms = t["dout"].double() * n2
        close(got["dnext_weight"], terms.sum(0), ((len(d) + 64) * U + FP) * terms.abs().sum(0) + 1e-30, "dnext_weight")
    else:
        dh = d
        assert got["dnext_weight"] is None
    close(got["dresidual"], dh, HALF[rtype] * dh.abs() + off_dh + 1e-30, "dresidual")
    a, slope, slope_size = (1, None, None) if z is None else gate(z)
    u = x * a
    w = t["w"].double()
    du, size, n, r = norm_bwd(SCALE * dh, u, w, EPS)
    off_p = SCALE * w.abs() * off_dh
    off_du = FP * size + r * (off_p + n.abs() * mean(n.abs() * off_p))
    dx = du * a
    close(got["dx"], dx, HALF[dtype] * dx.abs() + off_du * (a if z is None else a.abs()) + 1e-30, "dx")
    if z is None:
        assert got["dgate"] is None
    else:
        dz = du * x * slope
        close(got["dgate"], dz, HALF[dtype] * dz.abs() + (off_du + FP * size) * x.abs() * slope_size + 1e-30, "dgate")
    terms, off = SCALE * dh * n, SCALE * off_dh * n.abs()
    close(got["dweight"], terms.sum(0), ((len(d) + 64) * U + FP) * terms.abs().sum(0) + off.sum(0) + 1e-30, "dweight")


@pytest.mark.parametrize("rows,width,extra,offset", SHAPES)
@pytest.mark.parametrize("dtype,rtype", TYPES)
@pytest.mark.parametrize("gated,next_norm", [(True, True), (False, True), (True, False), (False, False)])
def test_gradient(rows, width, extra, offset, dtype, rtype, gated, next_norm):
    t = make(rows, width, dtype, rtype, rows + 3 * width, extra, offset, gated)
    h = t["res"] if next_norm else None
    whole = torch.full((rows, width + extra), 7.0, dtype=dtype, device="cuda") if gated else None
    got = ssd.block_norm_bwd(t["dout"] if next_norm else None, t["dres"], t["x"], h, t["w"], t["gate"], t["w2"] if next_norm else None,
                             scale=SCALE, eps=EPS, dgate=whole[:, :width] if gated else None)
    check(got, t, t["x"].double(), t["gate"].double() if gated else None, t["res"].double(), dtype, rtype, next_norm)
    assert not gated or (whole[:, width:] == 7).all()


@pytest.mark.parametrize("rows,width,extra,offset", SHAPES)
@pytest.mark.parametrize("dtype,rtype", TYPES)
@pytest.mark.parametrize("which", ["x", "gate", "h", "x gate h"])
def test_gradient_from_8_bit_rows(rows, width, extra, offset, dtype, rtype, which):
    gated = "gate" in which or rows % 2 == 1
    t = make(rows, width, dtype, rtype, rows + 5 * width, extra, offset, gated)
    args = {"x": t["x"], "gate": t["gate"], "h": t["res"]}
    kept = ssd.block_norm(t["x"], t["w"], t["res"], t["gate"], t["w2"], scale=SCALE, eps=EPS, pack=True)
    kept["h"], kept["h_scales"] = ssd.pack_rows(t["res"])
    for name in which.split():
        args[name], args[name + "_scales"] = kept[name], kept[name + "_scales"]
    got = ssd.block_norm_bwd(t["dout"], t["dres"], weight=t["w"], next_weight=t["w2"], scale=SCALE, eps=EPS, **args)
    value = lambda name: None if args[name] is None else wide(args[name], args.get(name + "_scales"))
    check(got, t, value("x"), value("gate"), value("h"), dtype, rtype, True)


def test_gradient_against_differences():
    t = make(6, 200, F4, F4, 11)
    f = ssd.block_norm(t["x"], t["w"], t["res"], t["gate"], t["w2"], scale=SCALE, eps=EPS)
    got = ssd.block_norm_bwd(t["dout"], t["dres"], t["x"], f["residual"], t["w"], t["gate"], t["w2"], scale=SCALE, eps=EPS)
    g = torch.Generator(device="cuda").manual_seed(5)
    names = {"x": "dx", "gate": "dgate", "res": "dresidual", "w": "dweight", "w2": "dnext_weight"}
    way = {k: torch.randn(t[k].shape, generator=g, device="cuda").double() for k in names}

    def value(step):
        _, h, _, out = formula({k: v.double() + step * way[k] if k in way else v for k, v in t.items()})
        return (out * t["dout"].double()).sum() + (h * t["dres"].double()).sum()

    slope = (value(1e-5) - value(-1e-5)) / 2e-5
    terms = torch.cat([(got[d].double() * way[k]).flatten() for k, d in names.items()])
    assert abs(terms.sum() - slope) <= 1e-5 * terms.abs().sum()


@pytest.mark.parametrize("width", [1283, 2560, 333, 64])
@pytest.mark.parametrize("packed", [False, True])
def test_rows_stay_apart(width, packed):
    t = make(912, width, BF, BF, width)

    def call():
        f = ssd.block_norm(t["x"], t["w"], t["res"], t["gate"], t["w2"], pack=packed)
        extra = {}
        x, z, h = t["x"], t["gate"], f["residual"]
        if packed:
            x, z, extra["x_scales"], extra["gate_scales"] = f["x"], f["gate"], f["x_scales"], f["gate_scales"]
            h, extra["h_scales"] = ssd.pack_rows(h)
        got = ssd.block_norm_bwd(t["dout"], t["dres"], x, h, t["w"], z, t["w2"], **extra)
        return {"h": f["residual"], "out": f["out"], **got}

    clean = call()
    t["dout"][5], t["x"][8], t["gate"][11, 3], t["res"][14, 0] = float("nan"), float("inf"), float("nan"), float("-inf")
    got = call()
    keep = torch.ones(912, dtype=torch.bool, device="cuda")
    keep[[5, 8, 11, 14]] = False
    for name in ("h", "out", "dx", "dgate", "dresidual"):
        assert torch.equal(got[name][keep], clean[name][keep]), name
    assert got["dweight"].isnan().all() and got["dnext_weight"].isnan().all()


def test_nothing_dimensions_stream_and_place():
    from mamba_ssd_chunked_scan_gb300 import _lib
    t = make(24, 136, BF, F4, 3)
    e = {k: v[:0] for k, v in t.items() if k not in ("w", "w2")}
    f = ssd.block_norm(e["x"], t["w"], e["res"], e["gate"], t["w2"], out_dtype=E4, pack=True)
    assert f["out"].shape == (0, 136) and f["scales"].shape == (0,) and f["gate_scales"].shape == (0,)
    got = ssd.block_norm_bwd(e["dout"], e["dres"], e["x"], e["res"], t["w"], e["gate"], t["w2"])
    assert (got["dweight"] == 0).all() and (got["dnext_weight"] == 0).all() and got["dgate"].shape == (0, 136)
    want = ssd.block_norm(t["x"], t["w"], t["res"], t["gate"], t["w2"], out_dtype=E4)
    back = ssd.block_norm_bwd(t["dout"], t["dres"], t["x"], t["res"], t["w"], t["gate"], t["w2"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    v = {k: x if k in ("w", "w2") else x.view(2, 3, 4, 136) for k, x in t.items()}
    f = ssd.block_norm(v["x"], t["w"], v["res"], v["gate"], t["w2"], out_dtype=E4, stream=s)
    b = ssd.block_norm_bwd(v["dout"], v["dres"], v["x"], v["res"], t["w"], v["gate"], t["w2"], stream=s)
    s.synchronize()
    assert f["scales"].shape == (2, 3, 4) and torch.equal(f["residual"].view(24, 136), want["residual"])
    assert torch.equal(f["out"].view(24, 136).view(torch.uint8), want["out"].view(torch.uint8))
    for k in back:
        assert torch.equal(b[k].flatten(), back[k].flatten())
    # residual_out may be the residual
    p = _lib.BlockNormParams(24, 136, 0, 136, 1, 0, 1, 1.0, 1e-5)
    res = t["res"].clone()
    rc = _lib.lib.ssd_block_norm(p, t["x"].data_ptr(), t["gate"].data_ptr(), res.data_ptr(), t["w"].data_ptr(), None, res.data_ptr(),
                                 *[None] * 6, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(res, want["residual"])


def test_refusals():
    t = make(4, 64, BF, F4, 1)
    f = ssd.block_norm(t["x"], t["w"], t["res"], t["gate"], t["w2"], pack=True)
    fwd = lambda **kw: ssd.block_norm(**{**dict(x=t["x"], weight=t["w"], residual=t["res"], gate=t["gate"], next_weight=t["w2"]), **kw})
    bwd = lambda **kw: ssd.block_norm_bwd(**{**dict(dout=t["dout"], dresidual=t["dres"], x=t["x"], h=t["res"], weight=t["w"], gate=t["gate"],
                                                    next_weight=t["w2"]), **kw})
    for bad in (lambda: fwd(x=t["x"].half()), lambda: fwd(residual=t["res"].half()), lambda: fwd(out_dtype=F4), lambda: fwd(x=t["x"].float(), residual=t["res"].to(BF)),
                lambda: bwd(dresidual=t["dres"].half()), lambda: bwd(dout=None, h=None, next_weight=None, x=f["x"], x_scales=f["x_scales"])):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: fwd(gate=t["gate"][:3]), lambda: fwd(gate=t["gate"].float()), lambda: fwd(weight=t["w"][:5]), lambda: fwd(next_weight=t["w2"].double()),
                lambda: fwd(x=t["x"].cpu()), lambda: bwd(dout=None), lambda: bwd(h=None), lambda: bwd(next_weight=None), lambda: bwd(x=f["x"]),
                lambda: bwd(x_scales=f["x_scales"]), lambda: bwd(gate=None, dgate=t["gate"]), lambda: bwd(gate_scales=f["gate_scales"]),
                lambda: bwd(gate=None, gate_scales=f["gate_scales"]), lambda: bwd(x=t["x"].t()), lambda: bwd(h=t["res"].to(BF)),
                lambda: bwd(x=torch.zeros(4, 128, dtype=BF, device="cuda")[:, :64])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fwd(eps=-1.0), lambda: fwd(scale=float("inf")), lambda: fwd(scale=float("nan")), lambda: bwd(dgate=t["gate"]), lambda: bwd(dgate=t["dout"])):
        with pytest.raises(ssd.SSDError):
            bad()
    big = torch.zeros(1, 8193, device="cuda")
    with pytest.raises(ssd.SSDError):
        ssd.block_norm(big, big[0], big)
