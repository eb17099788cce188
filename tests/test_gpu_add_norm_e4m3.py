"""The residual norm's 8-bit rows hold the quotient of the row and its scale, rounded once to fp32 and once to nearest even in
8 bits: values beside the midpoint of two neighbours go to the side that the division says.

Rows of ones and minus ones have a mean square of one exactly, so with eps = 0 the rows before the rounding are the weights
themselves, which the test places on midpoints and a few units of the last place off them."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn


@pytest.mark.parametrize("width", [24, 255, 512, 2560, 4099])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_midpoints_go_where_the_division_says(width, dtype):
    values = torch.arange(1, 127, dtype=torch.uint8).view(E4).float()   # every positive number below the largest
    mid = (values[1:] + values[:-1]) / 2
    gen = torch.Generator().manual_seed(width)
    for _ in range(40):
        amax = torch.exp2(torch.empty(()).uniform_(-12, 12, generator=gen))
        scale = amax / 448
        w = mid[torch.randint(len(mid), (width,), generator=gen)] * scale
        w = (w.view(torch.int32) + torch.randint(-2, 3, (width,), generator=gen, dtype=torch.int32)).view(torch.float32)
        sign = torch.randint(0, 2, (width,), generator=gen) * 2.0 - 1
        w[torch.randint(width, (1,), generator=gen)] = amax
        x = torch.stack([torch.ones(width), sign, -sign]).to(dtype).cuda()
        got = ssd.add_norm(x, w.cuda(), eps=0.0, out_dtype=E4)
        assert (got["scales"].cpu() == scale).all()
        want = (x.float().cpu() * w / scale).to(E4)
        assert torch.equal(got["out"].cpu().view(torch.uint8), want.view(torch.uint8))


def test_infinite_and_zero_rows():
    x = torch.ones(2, 40)
    x[1] = -1
    for big, other in ((float("inf"), 3.0), (3.0e38, 1e-3), (0.0, 0.0), (1e-30, 1e-32), (1e-37, -1e-38)):
        w = torch.full((40,), other)
        w[7] = big
        got = ssd.add_norm(x.cuda(), w.cuda(), eps=0.0, out_dtype=E4)
        scale = (x * w).abs().amax(1).clamp(min=1e-30) / 448
        want = (x * w / scale[:, None]).to(E4)
        assert torch.equal(got["scales"].cpu(), scale)
        a, b = got["out"].cpu().float(), want.float()
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
