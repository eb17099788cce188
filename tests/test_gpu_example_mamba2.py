"""The example's stack of Mamba-2 layers: norms, projections and scan together, with 8-bit checkpoints and without, against
automatic differentiation of the same formulas in 64 bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WEIGHTS = ("w_zx", "w_bc", "w_dt", "b_dt", "w_out", "A", "D", "gate", "post", "next")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("mamba2_layer", os.path.join(ROOT, "examples", "mamba2_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def norm(v, weight):
    return v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-5) * weight


def stack(layers, weights, first, s):
    """The same stack in 64 bits, differentiable."""
    n = norm(s, first)
    for l, w in zip(layers, weights):
        z, x = (n @ w["w_zx"].t()).chunk(2, -1)
        B, C = (n @ w["w_bc"].t() / l.state ** 0.5).chunk(2, -1)
        dt = torch.nn.functional.softplus(n @ w["w_dt"].t() + w["b_dt"])
        x = x.unflatten(-1, (l.heads, l.headdim))
        h, ys = 0, []
        for t in range(x.shape[1]):
            decay = torch.exp(dt[:, t] * w["A"])[..., None, None]
            h = decay * h + (dt[:, t, :, None] * x[:, t])[..., None] * B[:, t, None, None]
            ys.append((h * C[:, t, None, None]).sum(-1) + w["D"][:, None] * x[:, t])
        v = torch.stack(ys, 1).flatten(-2) * torch.nn.functional.silu(z)
        g = norm(v.unflatten(-1, (-1, l.group_size)), w["gate"].unflatten(-1, (-1, l.group_size))).flatten(-2)
        s = s + l.scale * norm(g @ w["w_out"].t(), w["post"])
        n = norm(s, w["next"])
    return n, s


# About twenty roundings to bf16 a layer lie on the way to any element, 2^-9 of the value at random each: 2 % after two layers.
# A's gradient sums differences of two sums of such terms.  With 8-bit checkpoints seven tensors a layer come from e4m3, off by 3 %
# at random each (up to 2^-4): 3 % sqrt(14), 11 % of the root of the sum of the terms' squares.  That root is the size of a sum
# of terms of random signs, too, but only on average: A, D and b_dt have four such sums, and of two sums of four squares one is
# 16 times the other in one case of a hundred (the F distribution), so that their errors' norm may reach four times 11 %.
@pytest.mark.parametrize("eight,tol,tol_a,tol_few", [(False, 0.05, 0.1, 0.05), (True, 0.2, 0.45, 0.45)])
@pytest.mark.parametrize("groups", [1, 2])
def test_gradients_against_automatic_differentiation(ex, eight, tol, tol_a, tol_few, groups):
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    layers = [ex.Layer(128, 4, gen, groups=groups) for _ in range(2)]
    first = torch.rand(128, generator=gen, device="cuda") + 0.5
    x, dn, ds = r(2, 150, 128), r(2, 150, 128).to(torch.bfloat16), r(2, 150, 128)
    weights = [{k: getattr(l, k).double().requires_grad_(True) for k in WEIGHTS} for l in layers]
    n, s = stack(layers, weights, first.double(), x.double())
    ((n * dn.double()).sum() + (s * ds.double()).sum()).backward()
    got_n, got_s, kept = ex.run(layers, first, x, eight)
    for got, want in ((got_n, n), (got_s, s)):
        assert ((got.double() - want).norm() / want.norm()) < 0.02
    for layer, saved, w in zip(reversed(layers), reversed(kept), reversed(weights)):
        dn, ds, grads = layer.backward(dn, ds, saved)
        assert set(grads) == set(WEIGHTS)
        for name, g in grads.items():
            off = ((g.double() - w[name].grad).norm() / w[name].grad.norm()).item()
            assert off < {"A": tol_a, "D": tol_few, "b_dt": tol_few}.get(name, tol), (name, off)


def test_gradients_from_8_bits_are_those_of_what_the_rows_stand_for(ex):
    """e4m3 times a power of two is exact in bf16: the same sums, in another order where a kernel of another shape takes them,
    which moves some of the roundings to bf16 by a step."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    layer, first = ex.Layer(128, 4, gen, groups=2), torch.ones(128, device="cuda")
    dn, ds = r(2, 150, 128).to(torch.bfloat16), r(2, 150, 128)
    tensors, dt, kept, block, s = ex.run([layer], first, r(2, 150, 128))[2][0]
    unpack = ex.ssd.unpack_rows
    plain = ([ex.Kept(k.tensor(), False) for k in tensors], dt, {k: unpack(kept[k], kept[k + "_scales"]) for k in ("y", "z")},
             {"x": unpack(block["x"], block["x_scales"])}, s)
    a, b = layer.backward(dn, ds, (tensors, dt, kept, block, s)), layer.backward(dn, ds, plain)
    for name, u, v in [("n", a[0], b[0]), ("s", a[1], b[1]), *[(k, a[2][k], b[2][k]) for k in WEIGHTS]]:
        assert ((u.double() - v.double()).norm() / v.double().norm()) < 2.0 ** -7, name


def test_the_checkpoint_leaves_the_forward_pass_and_is_smaller(ex):
    gen = torch.Generator(device="cuda").manual_seed(4)
    layers = [ex.Layer(256, 8, gen) for _ in range(2)]
    first, x = torch.ones(256, device="cuda"), torch.randn(2, 300, 256, generator=gen, device="cuda")
    a, b = ex.run(layers, first, x, True), ex.run(layers, first, x, False)
    for u, v in zip(a[:2], b[:2]):   # the gate and norm's sums differ in order, which moves some roundings to bf16 by a step
        assert ((u.double() - v.double()).norm() / v.double().norm()) < 2.0 ** -8
    eight, whole = (sum(ex.kept_bytes(k) for k in v[2]) for v in (a, b))
    assert eight < 0.65 * whole   # all but the fp32 stream and dt halve


def test_runs(ex):
    losses, sizes = ex.main(steps=2)
    assert all(torch.isfinite(torch.tensor(losses))) and sizes[0] < sizes[1]
