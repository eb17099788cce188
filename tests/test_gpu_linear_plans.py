"""The projection and its gradients on every way that a product is planned: tiles by a CTA or by a pair of them, transposed,
computed whole, in parts, or both in one launch, over several waves of tiles.  Each shape says which plan it stands for, and
the plan is asked whether it still does."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
import test_gpu_linear as base

pytestmark = pytest.mark.gpu

BF, E4 = torch.bfloat16, torch.float8_e4m3fn


def planned(m, n, k, kind, product=0):
    from mamba_ssd_chunked_scan_gb300 import _lib
    p = _lib.linear_plan(m, n, k, _lib.SSD_E4M3 if kind is E4 else _lib.SSD_BF16, product)
    what = "T" if p.transposed else "pair" if p.tile_rows == 256 else "cta"
    workers = 76 if what == "pair" else 152
    return "%s%d%s%s" % (what, p.tile_cols, " whole" if p.whole else "", " parts" if p.splits > 1 else ""), -(-p.tiles // workers)


# rows, columns, contraction, operands, plan, waves of tiles at least
FORWARD = [
    (8943, 1609, 2336, BF, "pair256 whole", 3), (6568, 1040, 4768, BF, "pair256 whole", 2),
    (5373, 2563, 2960, BF, "pair256 whole parts", 4), (6537, 1304, 4304, BF, "pair256 whole parts", 3),
    (2534, 7848, 4240, E4, "pair256 whole parts", 5), (4246, 3593, 4512, E4, "pair256 whole", 3),
    (1321, 3528, 1120, BF, "cta256 whole parts", 2), (6513, 1405, 1232, BF, "cta256 whole parts", 3),
    (789, 5520, 2192, E4, "cta256 whole parts", 2), (68, 6721, 5024, BF, "cta256 parts", 1),
    (292, 6412, 3920, BF, "cta128 whole parts", 2), (7741, 639, 3712, E4, "cta128 whole parts", 3), (141, 1276, 3088, BF, "cta128 parts", 1),
    (260, 6900, 16, BF, "cta64 whole", 3), (395, 7451, 16, E4, "cta128 whole", 2), (1426, 8088, 16, BF, "cta256 whole", 3),
    (9, 1001, 5120, E4, "T16 parts", 1), (24, 640, 5120, E4, "T32 parts", 1), (40, 1000, 5120, E4, "T64 parts", 1), (40, 1001, 2560, BF, "T64 parts", 1),
    (64, 20001, 64, BF, "T64 whole", 2),
]


@pytest.mark.parametrize("m,n,k,kind,plan,waves", FORWARD)
def test_forward_is_exact(m, n, k, kind, plan, waves):
    got = planned(m, n, k, kind)
    assert got[0] == plan and got[1] >= waves, got
    base.test_whole_numbers_are_exact(m, n, k, kind)


@pytest.mark.parametrize("m,n,k,kind,plan,waves", FORWARD)
@pytest.mark.parametrize("act,bias,res,pre", [("none", False, True, False), ("silu", True, True, True)])
def test_forward_with_its_epilogue(m, n, k, kind, plan, waves, act, bias, res, pre):
    base.test_forward(m, n, k, kind, act, bias, res, pre)


# rows, columns, contraction of the forward; the plans of dx and dw
GRADIENTS = [
    (7647, 7973, 528, "pair256 whole parts", "cta256 whole parts"), (3969, 3920, 2752, "pair256 whole parts", None),
    (7925, 3026, 1360, "pair256 whole", None), (3024, 8240, 1328, None, "pair256 whole"), (1503, 5846, 5072, None, "pair256 whole parts"),
    (1389, 1045, 3568, "cta256 whole parts", None), (1040, 1694, 2720, None, "cta256 whole parts"),
    (2155, 3653, 1056, "cta128 whole parts", None), (1758, 7770, 560, None, "cta128 whole parts"),
]


@pytest.mark.parametrize("m,n,k,dx,dw", GRADIENTS)
def test_gradients(m, n, k, dx, dw):
    for product, plan in ((1, dx), (2, dw)):
        if plan is not None:
            got = planned(m, n, k, BF, product)
            assert got[0] == plan, (product, got)
    base.test_whole_number_gradients_are_exact(m, n, k)
    base.test_gradients(m, n, k, "silu")


def test_repeats_itself():
    """Whole tiles and parts in one launch, the parts' sums joined: bit for bit the same each time."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    m, n, k = 5373, 2563, 2960
    x, w, res = r(m, k), r(n, k), r(m, n)
    want = ssd.linear(x, w, None, res)
    assert all(torch.equal(ssd.linear(x, w, None, res), want) for _ in range(5))
