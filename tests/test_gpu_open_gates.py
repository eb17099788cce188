"""Gates so far open that silu is the gate and its slope 1: the gradients of the norms after the scan and after a block against
the formulas in 64 bits, on vectors, shifted vectors and single elements, from tensors and from 8-bit rows.

From a gate of 30 on 1 / (1 + e^-z) is 1 in fp32 and silu's slope differs from 1 by 30 e^-30 < 2^-24, so the slope adds no error of its
own to dz beyond a product's rounding, which FP covers."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
from norms_helpers import BF, F4, FP, HALF, U, close, mean, norm_bwd, wide
from test_gpu_gate_norm_bwd import columns

pytestmark = pytest.mark.gpu

EPS = 1e-5
SIZES = [30.0, 300.0, 5000.0, 2.0 ** 24 + 2, 2.0 ** 25 + 4, 1e8, 3e10, 1e15]
# vectors by lanes and by CTAs, shifted ones, single elements (rows or buffers off 16 bytes)
SHAPES = [(64, 0, 0), (520, 8, 0), (2560, 0, 0), (37, 0, 0), (1283, 0, 0), (64, 3, 0), (520, 0, 1)]


def make(width, dtype, extra, offset, seed):
    """Rows whose gates are of one size each, so that no element rules its row."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = 2 * len(SIZES)
    size = torch.tensor(SIZES, device="cuda").repeat(2)[:, None]
    z = size * (1 + torch.rand(rows, width, generator=g, device="cuda"))
    y, d, e = (torch.randn(rows, width, generator=g, device="cuda") for _ in range(3))
    w = torch.rand(width, generator=g, device="cuda") + 0.5
    c = lambda v, x=0: columns(v.to(dtype), x, offset)
    return c(y), c(z, extra), c(d), c(e), w


def check(got, dx, dgate, p, x, z, w, dtype):
    """p: the gradient of the norm's result; silu(z) is z and its slope 1."""
    u = x * z
    du, size, _, _ = norm_bwd(p, u, w.double(), EPS)
    want = du * x
    close(got[dgate], want, HALF[dtype] * want.abs() + 2 * FP * size * x.abs() + 1e-36, dgate)
    want = du * z
    close(got[dx], want, HALF[dtype] * want.abs() + FP * size * z.abs() + 1e-36, dx)


@pytest.mark.parametrize("width,extra,offset", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F4])
@pytest.mark.parametrize("packed", [False, True])
def test_gate_and_norm(width, extra, offset, dtype, packed):
    y, z, d, _, w = make(width, dtype, extra, offset, width)
    args = dict(y=y, z=z)
    if packed:
        args = ssd.gate_norm(y, z, w, width, EPS, pack=True)[1]
        if offset:
            args["y"] = columns(args["y"].view(torch.uint8), 0, 1).view(args["y"].dtype)
    got = ssd.gate_norm_bwd(d, weight=w, group_size=width, eps=EPS, want_out=True, **args)
    x, gate = wide(args["y"], args.get("y_scales")), wide(args["z"], args.get("z_scales"))
    check(got, "dy", "dz", d.double(), x, gate, w, dtype)
    u = x * gate
    out = u * torch.rsqrt(mean(u * u) + EPS) * w.double()
    close(got["out"], out, (HALF[dtype] + FP) * out.abs() + 1e-36, "out")


@pytest.mark.parametrize("width,extra,offset", SHAPES)
@pytest.mark.parametrize("dtype,rtype", [(BF, F4), (BF, BF), (F4, F4)])
@pytest.mark.parametrize("packed", [False, True])
def test_norm_after_a_block(width, extra, offset, dtype, rtype, packed):
    x, z, _, e, w = make(width, dtype, extra, offset, 3 * width)
    dres = columns(e.to(rtype), 0, offset)
    args = dict(x=x, gate=z)
    if packed:
        f = ssd.block_norm(x, w, torch.zeros_like(dres), z, scale=0.5, eps=EPS, pack=True)
        args = {k: f[k] for k in ("x", "x_scales", "gate", "gate_scales")}
        if offset:
            args["x"] = columns(args["x"].view(torch.uint8), 0, 1).view(args["x"].dtype)
    got = ssd.block_norm_bwd(None, dres, h=None, weight=w, scale=0.5, eps=EPS, dtype=dtype, **args)
    check(got, "dx", "dgate", 0.5 * dres.double(), wide(args["x"], args.get("x_scales")), wide(args["gate"], args.get("gate_scales")), w, dtype)


@pytest.mark.parametrize("dtype", [BF, F4])
def test_moderate_gates_keep_the_slope(dtype):
    """Gates of 17 to 30, where 1 - 1 / (1 + e^-z) goes below fp32's steps: the slope is 1 + z e^-z to within z 2^-24."""
    g = torch.Generator(device="cuda").manual_seed(2)
    z = (torch.rand(40, 512, generator=g, device="cuda") * 13 + 17).to(dtype)
    y, d = (torch.randn(40, 512, generator=g, device="cuda").to(dtype) for _ in range(2))
    w = torch.rand(512, generator=g, device="cuda") + 0.5
    got = ssd.gate_norm_bwd(d, y, z, w, 512, EPS)
    zd, yd = z.double(), y.double()
    s = torch.sigmoid(zd)
    a = zd * s
    du, size, _, _ = norm_bwd(d.double(), yd * a, w.double(), EPS)
    want = du * yd * (s + a * (1 - s))
    # 1 / (1 + e^-z) is off by U of the sum and 2 U of the quotient (rcp.approx; a division U / 2), which z multiplies
    close(got["dz"], want, HALF[dtype] * want.abs() + (2 * FP * size + du.abs() * zd * 3 * U) * yd.abs() + 1e-36, "dz")
