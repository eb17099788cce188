"""The activations' slopes at the largest arguments of their type and at infinities: one where the activation follows its
argument, zero where it is flat, and NaN only for NaN."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_slopes_at_the_limits(act):
    far = [1e3, 1e10, 1e15, 1e20, torch.finfo(BF).max, float("inf")]
    pre = torch.tensor([far + [-v for v in far] + [float("nan"), 0.0, 1.0, -1.0]], device="cuda").to(BF)
    n = pre.shape[1]
    dy = torch.full((1, n), 3.0, dtype=BF, device="cuda")
    x, w = torch.ones(1, 8, dtype=BF, device="cuda"), torch.zeros(n, 8, dtype=BF, device="cuda")
    got = ssd.linear_bwd(dy, x, w, pre, act=act, want_dbias=True)
    k = len(far)
    for g in (got["dbias"], got["dw"][:, 0].float()):
        assert (g[:k] == 3).all() and (g[k:2 * k] == 0).all() and g[2 * k].isnan(), g
        assert torch.isfinite(g[2 * k + 1:]).all() and (g[2 * k + 1] == 1.5).all()
    # slopes between, against automatic differentiation in 64 bits
    v = torch.linspace(-30, 30, 16 * 512, device="cuda").to(BF).view(512, 16)
    d = v.double().requires_grad_(True)
    f = torch.nn.functional.silu(d) if act == "silu" else torch.nn.functional.gelu(d, approximate="tanh")
    want = torch.autograd.grad(f.sum(), d)[0]
    got = ssd.linear_bwd(torch.ones_like(v), torch.ones(512, 8, dtype=BF, device="cuda"), torch.zeros(16, 8, dtype=BF, device="cuda"), v,
                         act=act, want_dx=False, want_dw=False, want_dbias=True)
    assert (got["dbias"].double() - want.sum(0)).abs().max() <= 512 * 64 * 2.0 ** -24 * 1.2
