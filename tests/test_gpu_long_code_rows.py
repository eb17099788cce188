"""Long rows of 8-bit codes with large gates in the norms' gradients: sums are of what the codes stand for."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
from norms_helpers import BF, F4, wide
from test_gpu_open_gates import EPS, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["gate and norm", "norm after a block"])
@pytest.mark.parametrize("dtype", [BF, F4])
def test_long_rows_of_codes(which, dtype):
    """8192 codes times gates of 1e15: their squares' sum passes fp32's largest number before the scale joins it, that of what the
    codes stand for does not."""
    g = torch.Generator(device="cuda").manual_seed(4)
    rows, width = 5, 8192
    sign = torch.randint(0, 2, (rows, width), generator=g, device="cuda") * 2 - 1
    x = ((1 + torch.rand(rows, width, generator=g, device="cuda") * 0.75) * sign).to(dtype)
    z = (1e15 * (1 + torch.rand(rows, width, generator=g, device="cuda"))).to(dtype)
    d = torch.randn(rows, width, generator=g, device="cuda").to(dtype)
    w = torch.rand(width, generator=g, device="cuda") + 0.5
    (xq, xs), (zq, zs) = ssd.pack_rows(x), ssd.pack_rows(z)
    if which == "gate and norm":
        got = ssd.gate_norm_bwd(d, xq, zq, w, width, EPS, y_scales=xs[:, None], z_scales=zs[:, None])
        check(got, "dy", "dz", d.double(), wide(xq, xs), wide(zq, zs), w, dtype)
    else:
        got = ssd.block_norm_bwd(None, d, xq, None, w, zq, scale=0.5, eps=EPS, x_scales=xs, gate_scales=zs, dtype=dtype)
        check(got, "dx", "dgate", 0.5 * d.double(), wide(xq, xs), wide(zq, zs), w, dtype)
