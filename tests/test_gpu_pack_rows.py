"""8-bit rows on the GPU against a table of every e4m3 number: all of it is exact."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
from norms_helpers import BF, E4, F4, rows_by_table, same_codes, wide

pytestmark = pytest.mark.gpu


def make(rows, width, dtype, seed, extra=0, offset=0):
    """Rows of very different sizes, zeros among them; with `extra`, columns of a wider matrix; `offset` elements into a buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.zeros(rows * (width + extra) + offset, dtype=dtype, device="cuda")
    x = flat[offset:].view(rows, width + extra)[:, :width]
    v = torch.randn(rows, width, generator=g, device="cuda")
    v *= torch.exp2(torch.randint(-60, 60, (rows, 1), generator=g, device="cuda").float())
    v *= torch.exp2(torch.randint(-12, 1, (rows, width), generator=g, device="cuda").float())   # down to the subnormals
    v[torch.rand(rows, generator=g, device="cuda") < 0.1] = 0
    x.copy_(v)
    return x


SHAPES = [(1, 1, 1), (3, 7, 1), (5, 24, 3), (2, 512, 1), (9, 513, 1), (33, 640, 5), (17, 2557, 1), (40, 2560, 1), (6, 5120, 80), (3, 8192, 1),
          (2, 16384, 1), (2, 16383, 3), (1, 32768, 2)]


@pytest.mark.parametrize("rows,width,groups", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F4])
@pytest.mark.parametrize("extra,offset", [(0, 0), (16, 0), (3, 0), (0, 1)])
def test_codes_and_scales(rows, width, groups, dtype, extra, offset):
    x = make(rows, width, dtype, rows + width, extra, offset)
    codes, scales = ssd.pack_rows(x, width // groups)
    want, per = rows_by_table(x, groups)
    assert torch.equal(scales.cpu(), per) and same_codes(codes, want)
    if groups == 1:
        again, one = ssd.pack_rows(x)
        assert one.shape == (rows,) and torch.equal(one, scales[:, 0]) and torch.equal(again.view(torch.uint8), codes.view(torch.uint8))
    for kind in (BF, F4):   # exact in both types
        back = ssd.unpack_rows(codes, scales, dtype=kind)
        assert back.dtype is kind and torch.equal(back.double(), wide(codes, scales))


@pytest.mark.parametrize("dtype", [BF, F4])
def test_midpoints_and_borders(dtype):
    """Every value between two neighbouring e4m3 numbers, and beside it; the largest magnitudes on both sides of a power of two's 448."""
    number = torch.arange(127, dtype=torch.uint8).view(E4).double()
    mid = (number[:-1] + number[1:]) / 2
    beside = torch.cat([mid, torch.nextafter(mid.float(), torch.tensor(1e9)).double(), torch.nextafter(mid.float(), torch.tensor(0.0)).double()])
    rows = torch.stack([torch.cat([beside, -beside, torch.tensor([448.0 * f])]) * s for f in (1, 0.75, 0.57) for s in (1.0, 2.0 ** 40, 2.0 ** -50)])
    x = rows.to(dtype).cuda()
    codes, scales = ssd.pack_rows(x)
    want, per = rows_by_table(x)
    assert torch.equal(scales.cpu(), per[:, 0]) and same_codes(codes, want)
    tops = torch.tensor([448.0, 449.0, 450.0, 447.0, 224.0, 225.0, 3.0e38, 1e-37, 2.0 ** -126, 1e-40, 2.0 ** -100, 448 * 2.0 ** -108, 0.0]).to(dtype)
    x = tops[:, None].cuda().expand(-1, 40).contiguous()
    codes, scales = ssd.pack_rows(x)
    want, per = rows_by_table(x)
    assert torch.equal(scales.cpu(), per[:, 0]) and same_codes(codes, want)


@pytest.mark.parametrize("width", [5, 40, 513, 1024, 2560])
@pytest.mark.parametrize("dtype", [BF, F4])
def test_infinities_and_nans_stay_alone(width, dtype):
    x = make(7, width, dtype, width)
    x[1, 2], x[2, 3], x[3, 0], x[3, 4] = float("inf"), float("nan"), float("-inf"), float("nan")
    x[5] = float("nan")
    x[6] = float("inf")
    codes, scales = ssd.pack_rows(x)
    want, per = rows_by_table(x)
    assert torch.equal(scales.cpu(), per[:, 0]) and same_codes(codes, want)
    assert torch.equal(ssd.unpack_rows(codes, scales).isnan(), ~x.isfinite())


def test_unpack_of_other_scales():
    """Scales that are no powers of two (add_norm's): rounded once."""
    x = torch.randn(50, 203, device="cuda")
    n = ssd.add_norm(x, torch.ones(203, device="cuda"), out_dtype=E4)
    exact = wide(n["out"], n["scales"])
    assert torch.equal(ssd.unpack_rows(n["out"], n["scales"], dtype=F4), exact.float())
    bf = ssd.unpack_rows(n["out"], n["scales"])
    assert torch.equal(bf, exact.float().to(BF))   # an fp32 product of 4 and 24 bits rounds first: 2^-24 of it


def test_dimensions_and_nothing():
    x = torch.randn(2, 3, 48, device="cuda")
    codes, scales = ssd.pack_rows(x)
    assert codes.shape == (2, 3, 48) and scales.shape == (2, 3)
    codes, scales = ssd.pack_rows(x, 16)
    assert scales.shape == (2, 3, 3) and ssd.unpack_rows(codes, scales).shape == (2, 3, 48)
    codes, scales = ssd.pack_rows(x[:0])
    assert codes.shape == (0, 3, 48) and scales.shape == (0, 3) and ssd.unpack_rows(codes, scales).shape == (0, 3, 48)
    one, s = ssd.pack_rows(x[0, 0])
    assert one.shape == (48,) and s.shape == ()


def test_refusals():
    x = torch.randn(4, 64, device="cuda")
    for bad in (lambda: ssd.pack_rows(x.half()), lambda: ssd.unpack_rows(*ssd.pack_rows(x), dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    codes, scales = ssd.pack_rows(x)
    for bad in (lambda: ssd.pack_rows(x.cpu()), lambda: ssd.pack_rows(x, 48), lambda: ssd.pack_rows(x, 0), lambda: ssd.pack_rows(x[:, ::2]),
                lambda: ssd.pack_rows(x.t()), lambda: ssd.unpack_rows(x, scales), lambda: ssd.unpack_rows(codes, scales[:3]),
                lambda: ssd.unpack_rows(codes, scales.double()), lambda: ssd.unpack_rows(codes[:, :32], scales),
                lambda: ssd.unpack_rows(codes, torch.ones(4, 5, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ssd.SSDError):
        ssd.pack_rows(torch.zeros(1, 16385, device="cuda"))
