"""The norms around a block where each slot of the grid takes many rows one after another: every row, and the sums over all of them,
against the formulas in 64 bits.

Forwards a slot takes up to 8 rows through two stages of shared memory, backwards as many as there are.  GPU's slots: 152 SMs times the
CTAs an SM holds times a CTA's slots (16, 8 or 4 of 8, 16 or 32 lanes up to 256 columns, else one)."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
import test_gpu_block_norm as B
import test_gpu_gate_norm_bwd as G
from norms_helpers import BF, E4, F4, FP, HALF, U, close, gate, mean, norm_bwd, wide

pytestmark = pytest.mark.gpu

EPS, SCALE = B.EPS, B.SCALE
# rows, width, columns between rows of the gate: two, three and eight rows a slot and some left over; CTAs of 16 and of 8 elements a
# thread, lanes, each with rows of whole vectors and without
SHAPES = [(1221, 2560, 80), (1831, 2560, 0), (5003, 2560, 0), (1523, 1533, 0), (6101, 1533, 0), (3045, 520, 8), (12203, 765, 0), (34101, 64, 0),
          (34133, 37, 0), (17101, 128, 8), (8609, 245, 0), (8533, 256, 0)]


def bits(t):
    return t.contiguous().view(torch.uint8)


def same_rows(got, name, x, groups=1):
    codes, scales = ssd.pack_rows(x, x.shape[-1] // groups)
    assert torch.equal(bits(got[name]), bits(codes)) and torch.equal(got[name + "_scales"].flatten(), scales.flatten()), name


@pytest.mark.parametrize("rows,width,extra", SHAPES)
@pytest.mark.parametrize("dtype,rtype", B.TYPES)
@pytest.mark.parametrize("gated,out_dtype,pack", [(True, None, True), (False, E4, False), (True, E4, True), (False, None, True)])
def test_norm_after_a_block(rows, width, extra, dtype, rtype, gated, out_dtype, pack):
    t = B.make(rows, width, dtype, rtype, rows + width, extra, 0, gated)
    got = ssd.block_norm(t["x"], t["w"], t["res"], t["gate"], t["w2"], scale=SCALE, eps=EPS, out_dtype=out_dtype, pack=pack)
    n, h, r2, out = B.formula(t)
    off_h = FP * n.abs() + 2 * U * h.abs()
    close(got["residual"], h, HALF[rtype] * h.abs() + off_h + 1e-30, "residual")
    off = FP * out.abs() + r2 * t["w2"].double().abs() * off_h + out.abs() * r2 * r2 * mean(h.abs() * off_h)
    if out_dtype is E4:
        s = got["scales"].double()[:, None]
        top = out.abs().amax(1, keepdim=True)
        assert ((448 * s >= top * (1 - 4 * FP)) & (224 * s < top * (1 + 4 * FP))).all()
        close(wide(got["out"], got["scales"]), out, 2.0 ** -4 * out.abs() + 2.0 ** -10 * s + 2 * off, "e4m3")
    else:
        close(got["out"], out, HALF[dtype] * out.abs() + off + 1e-30, "out")
    if pack:
        same_rows(got, "x", t["x"])
        if gated:
            same_rows(got, "gate", t["gate"])
    one = ssd.block_norm(t["x"], t["w"], t["res"], t["gate"], scale=SCALE, eps=EPS)   # no next norm: one sum a row
    assert torch.equal(one["residual"], got["residual"])


GROUPED = [*[(r, w, 1, e) for r, w, e in SHAPES], (3101, 5120, 80, 16), (6005, 1536, 3, 0), (12007, 111, 3, 0), (2011, 5120, 8, 80)]


@pytest.mark.parametrize("rows,width,groups,extra", GROUPED)
@pytest.mark.parametrize("dtype", [BF, F4])
def test_gate_and_norm(rows, width, groups, extra, dtype):
    y, z, _, w = G.make(rows, width, dtype, rows + width, extra)
    out, kept = ssd.gate_norm(y, z, w, width // groups, EPS, pack=True)
    u = y.double() * gate(z.double())[0]
    want = u * torch.rsqrt(mean(u * u, groups) + EPS) * w.double()
    close(out, want, (HALF[dtype] + FP) * want.abs() + 1e-30, "out")
    same_rows(kept, "y", y, groups)
    same_rows(kept, "z", z, groups)


def sums(got, terms, off=0):
    """A weight's gradient: the rows of a slot one after another (of at least 152 CTAs of at least 4 slots where rows are 245 columns
    or less), then the slots' shares, up to 24320 by 64 threads and these in turn."""
    rows, width = terms.shape
    chain = rows / (152 * (4 if width <= 245 else 1)) + 24320 / 64 + 64
    close(got, terms.sum(0), (chain * U + FP) * terms.abs().sum(0) + off + 1e-30, "a weight's gradient")


@pytest.mark.parametrize("rows,width,groups,extra", GROUPED)
@pytest.mark.parametrize("dtype", [BF, F4])
@pytest.mark.parametrize("packed", [False, True])
def test_gate_and_norm_gradient(rows, width, groups, extra, dtype, packed):
    y, z, d, w = G.make(rows, width, dtype, rows + 3 * width, 0 if packed else extra)
    args = ssd.gate_norm(y, z, w, width // groups, EPS, pack=True)[1] if packed else dict(y=y, z=z)
    whole = torch.full((rows, width + extra), 7.0, dtype=dtype, device="cuda")
    got = ssd.gate_norm_bwd(d, weight=w, group_size=width // groups, eps=EPS, dz=whole[:, :width], want_out=True, **args)
    y, z = wide(args["y"], args.get("y_scales")), wide(args["z"], args.get("z_scales"))
    G.check(got, d, y, z, w, groups, dtype, True)
    u = y * gate(z)[0]
    sums(got["dweight"], d.double() * u * torch.rsqrt(mean(u * u, groups) + EPS))
    assert (whole[:, width:] == 7).all()


# The last rows are left to further slots from 16 rows a slot on: bf16 from tensors.  Just below, at and above that.
LATE = [(2560, 1, 9728), (5120, 80, 2432), (1536, 3, 8064), (37, 1, 194560), (515, 1, 24320), (128, 1, 97280)]


@pytest.mark.parametrize("width,groups,rows", [(w, g, r + k) for w, g, r in LATE for k in (-1, 0, 5)])
def test_gate_and_norm_gradient_with_late_slots(width, groups, rows):
    """dout holds a few columns a row, so that each column's sum is of few rows and one that is left out, or taken twice, shows."""
    y, z, d, w = G.make(rows, width, BF, rows)
    where = torch.randint(0, width, (rows, 4), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    d = d * torch.zeros_like(d).scatter_(1, where, 1.0)
    got = ssd.gate_norm_bwd(d, y, z, w, width // groups, EPS, want_out=True)
    G.check(got, d, y.double(), z.double(), w, groups, BF, True)
    u = y.double() * gate(z.double())[0]
    sums(got["dweight"], d.double() * u * torch.rsqrt(mean(u * u, groups) + EPS))
    again = ssd.gate_norm_bwd(d, y, z, w, width // groups, EPS)
    assert all(torch.equal(again[k], got[k]) for k in ("dy", "dz", "dweight"))


@pytest.mark.parametrize("rows,width,extra", SHAPES)
@pytest.mark.parametrize("dtype,rtype", B.TYPES)
@pytest.mark.parametrize("gated,next_norm", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("packed", [False, True])
def test_norm_after_a_block_gradient(rows, width, extra, dtype, rtype, gated, next_norm, packed):
    t = B.make(rows, width, dtype, rtype, rows + 3 * width, 0 if packed else extra, 0, gated)
    args = dict(x=t["x"], gate=t["gate"], h=t["res"] if next_norm else None)
    if packed:
        f = ssd.block_norm(t["x"], t["w"], t["res"], t["gate"], scale=SCALE, eps=EPS, pack=True)
        args = {k: f[k] for k in ("x", "x_scales", "gate", "gate_scales")}
        args["h"], args["h_scales"] = ssd.pack_rows(t["res"]) if next_norm else (None, None)
    got = ssd.block_norm_bwd(t["dout"] if next_norm else None, t["dres"], weight=t["w"], next_weight=t["w2"] if next_norm else None, scale=SCALE, eps=EPS,
                             dtype=dtype, **args)
    value = lambda k: None if args[k] is None else wide(args[k], args.get(k + "_scales"))
    x, z, h = value("x"), value("gate"), value("h")
    B.check(got, t, x, z, h, dtype, rtype, next_norm)
    dh, off = t["dres"].double(), 0
    if next_norm:
        back, size, n2, _ = norm_bwd(t["dout"].double(), h, t["w2"].double(), EPS)
        dh, off = dh + back, FP * size
        sums(got["dnext_weight"], t["dout"].double() * n2)
    u = x if z is None else x * gate(z)[0]
    n = u * torch.rsqrt(mean(u * u) + EPS)
    sums(got["dweight"], SCALE * dh * n, (SCALE * (off + 4 * U * dh.abs()) * n.abs()).sum(0))
