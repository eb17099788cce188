"""The recurrence's gradient where inputs hardly move and gates are nearly open, so that h lies close to x.

The backward pass reads h at every few tokens from y, in y's type (include/ssd.h says so).  The gradient of g holds the
difference h_{t-1} - x_t, which keeps the absolute error of that rounding: dg is off by up to
|lam| a (1 - a) 2^-8 |h| in bf16, however small the difference is, and by fp32's rounding with fp32 tensors."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
from test_gpu_gate_scan import BF, F4, OUT, U, walk, walk_back

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqlen,width", [(700, 64), (700, 61), (3000, 128)])
@pytest.mark.parametrize("dtype", [BF, F4])
@pytest.mark.parametrize("gate", [0.5, 3.0, 8.0])
def test_inputs_that_hardly_move(seqlen, width, dtype, gate):
    gen = torch.Generator(device="cuda").manual_seed(seqlen + width)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    level = r(1, 1, width) + 3
    x = (level + 1e-3 * r(1, seqlen, width)).to(dtype)
    g, dy, init = (r(1, seqlen, width) * 0.1 + gate).to(dtype), r(1, seqlen, width).to(dtype), level[:, 0].contiguous()
    y = ssd.gate_scan(g, x, init, check_status=True)
    got = ssd.gate_scan_bwd(g, x, y, dy, init, check_status=True)
    a, m, h, before, H, E = walk(g, x, init, None)
    lam, Lm, EL, mu, Em = walk_back(g, a, dy, None, None)
    dg = lam * (before - x.double()) * a * m
    # h read from y, off by its rounding and its own error; two gate roundings and the adjoint's error on the small difference
    eh = torch.cat([torch.zeros_like(E[:, :1]), E[:, :-1] + OUT[dtype] * (H + E)[:, :-1]], 1) + 2 * U * (before.abs() + x.double().abs())
    near = (before - x.double()).abs() * a * m
    bound = OUT[dtype] * dg.abs() + Lm * a * m * eh + (EL + U * (16 + 8 * g.double().abs()) * Lm) * (near + a * m * eh)
    worst = ((got["dg"].double() - dg).abs() / (bound + 1e-30)).max().item()
    assert worst <= 1, worst
