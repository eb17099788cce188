"""The gated recurrence where gates close: decays far below the rounding of one keep their own precision.

Bounds.  With U = 2^-24: a = 1 / (1 + exp(-g)) carries the rounding of the exponential's argument (|g| log2 e, and its
constant's own), 2^-22 of the exponential, 2^-23 of the reciprocal and a sum's U: U (7 + 1.25 |g|) of its value, whatever
the value is.  A step and the composition of maps round a handful of times more.  So with x = 0 a state, a product of decays, is
within the sum of U (12 + 2 |g_t|) of its own value, and the initial states' gradient a_1 lam_1 within U (12 + 4 |g_1|) of
a_1 times the magnitudes behind lam_1; nothing is measured against the state or the adjoint before it decayed.  Outputs of
16 bits round once more."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
from test_gpu_gate_scan import BF, F4, OUT, U, offsets, walk

pytestmark = pytest.mark.gpu

FLOOR = 1e-35   # below this fp32 has no full precision of its own


def near(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    worst = ((got.double() - want).abs() / (bound + FLOOR)).max().item()
    assert worst <= 1, (what, worst)


def closing(batch, seqlen, width, dtype, seed, places):
    """Gates that forget nearly nothing but at up to two tokens of each row, where logits run from -25 to -8 over the channels."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    g = torch.full((batch, seqlen, width), 20.0, device="cuda")
    ramp = -25 + 17 * torch.rand(width, generator=gen, device="cuda")
    for b in range(batch):
        for t in places[b % len(places)]:
            g[b, t % seqlen] = ramp.roll(t)
    return g.to(dtype), r


def mags(a, g, dy, dfin, ends):
    """lam, its magnitudes and its error, as the decays and not one minus them make them."""
    L, z = dy.shape[1], torch.zeros_like(dy[:, 0])
    lam, Lm, E = (torch.zeros_like(dy) for _ in range(3))
    mu = Mm = Em = z
    for t in range(L - 1, -1, -1):
        if t in ends:
            mu = dfin if ends[t] is None else dfin[ends[t]][None]
            Mm, Em = mu.abs(), z
        lam[:, t], Lm[:, t] = dy[:, t] + mu, dy[:, t].abs() + Mm
        E[:, t] = Em + 2 * U * Lm[:, t]
        mu, Mm = a[:, t] * lam[:, t], a[:, t] * Lm[:, t]
        Em = a[:, t] * E[:, t] + U * (12 + 4 * g[:, t].abs()) * Mm
    return lam, Lm, E, mu, Em


PLACES = [(0,), (1,), (7, 130), (15, 16), (0, -1), (127, 128), (255, 256), (-1,), (300, 301)]
SHAPES = [(1, 1, 40), (9, 70, 64), (9, 700, 64), (9, 700, 61), (2, 2100, 128)]


@pytest.mark.parametrize("batch,seqlen,width", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F4])
def test_states_decay_to_their_own_value(batch, seqlen, width, dtype):
    g, r = closing(batch, seqlen, width, dtype, seqlen + width, PLACES)
    x, init = torch.zeros_like(g), r(batch, width) * 100
    y, fin = ssd.gate_scan(g, x, init, return_final_states=True, check_status=True)
    gd = g.double()
    h = init.double()[:, None] * torch.sigmoid(gd).cumprod(1)
    rel = (U * (12 + 2 * gd.abs())).cumsum(1)
    near(fin, h[:, -1], rel[:, -1] * h[:, -1].abs(), "final states")
    near(y, h, (rel + OUT[dtype]) * h.abs(), "y")
    # the same tokens one by one
    state = init.clone()
    for t in range(min(seqlen, 20)):
        out = ssd.gate_scan_step(state, g[:, t].contiguous(), x[:, t].contiguous())
        near(out, h[:, t], (rel[:, t] + OUT[dtype]) * h[:, t].abs(), "step")


@pytest.mark.parametrize("batch,seqlen,width", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F4])
def test_large_states_are_forgotten(batch, seqlen, width, dtype):
    g, r = closing(batch, seqlen, width, dtype, 2 * seqlen + width, PLACES)
    x, init = (r(batch, seqlen, width) * 1e-3).to(dtype), r(batch, width) * 1e6
    y, fin = ssd.gate_scan(g, x, init, return_final_states=True, check_status=True)
    a, m, h, before, H, E = walk(g, x, init, None)
    near(y, h, OUT[dtype] * h.abs() + E, "y")
    near(fin, h[:, -1], E[:, -1], "final states")


@pytest.mark.parametrize("batch,seqlen,width", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F4])
def test_gradients_through_closed_gates(batch, seqlen, width, dtype):
    g, r = closing(batch, seqlen, width, dtype, 3 * seqlen + width, PLACES)
    x, init, dy, dfin = r(batch, seqlen, width).to(dtype), r(batch, width), r(batch, seqlen, width).to(dtype), r(batch, width)
    y = ssd.gate_scan(g, x, init, check_status=True)
    got = ssd.gate_scan_bwd(g, x, y, dy, init, dfin, check_status=True)
    gd = g.double()
    a, m = torch.sigmoid(gd), torch.sigmoid(-gd)
    lam, Lm, E, mu, Em = mags(a, gd, dy.double(), dfin.double(), {seqlen - 1: None})
    near(got["dinit"], mu, Em, "dinit")
    gate = U * (8 + 4 * gd.abs())
    near(got["dx"], m * lam, OUT[dtype] * (m * lam).abs() + m * E + gate * m * Lm, "dx")


def test_documents_first_gates_closed():
    lens = [1, 130, 3, 700, 16, 64]
    for dtype in (BF, F4):
        for width in (64, 61):
            gen = torch.Generator(device="cuda").manual_seed(width)
            r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
            cu, n, L = offsets(lens), len(lens), sum(lens)
            g = torch.full((1, L, width), 20.0, device="cuda")
            first = cu.tolist()[:-1]
            g[0, first] = -25 + 17 * torch.rand(n, width, generator=gen, device="cuda")
            g, x, dy, init, dfin = g.to(dtype), torch.zeros(1, L, width, device="cuda").to(dtype), r(1, L, width).to(dtype), r(n, width), r(n, width)
            y, fin = ssd.gate_scan(g, x, init, cu, return_final_states=True, check_status=True)
            got = ssd.gate_scan_bwd(g, x, y, dy, init, dfin, cu, check_status=True)
            gd = g.double()
            a = torch.sigmoid(gd)
            for d in range(n):
                s = slice(first[d], first[d] + lens[d])
                h = init[d].double() * a[0, s].cumprod(0)
                rel = (U * (12 + 2 * gd[0, s].abs())).cumsum(0)
                near(y[0, s], h, (rel + OUT[dtype]) * h.abs(), "y")
                near(fin[d], h[-1], rel[-1] * h[-1].abs(), "final states")
            ends = {t - 1: d for d, t in enumerate(cu.tolist()[1:])}
            lam, Lm, E, mu, Em = mags(a, gd, dy.double(), dfin.double(), ends)
            near(got["dinit"], (a * lam)[0, first], (a * E + U * (12 + 4 * gd.abs()) * a * Lm)[0, first], "dinit")
