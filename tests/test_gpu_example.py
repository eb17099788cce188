"""The example's stack of gated layers: its gradients against automatic differentiation of the same formulas in 64 bits,
its training, and its decoding against its prefill."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("gated_block", os.path.join(ROOT, "examples", "gated_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def stack(layers, d):
    """The same stack in 64 bits, differentiable."""
    s = torch.zeros_like(d)
    for w in layers:
        s = d + s
        n = s / torch.sqrt(s.square().mean(-1, keepdim=True) + 1e-5) * w["norm"]
        g, x = (n @ w["w_in"].t() + w["b_in"]).chunk(2, -1)
        h, hs = torch.zeros_like(g[:, 0]), []
        for t in range(g.shape[1]):
            h = torch.sigmoid(g[:, t]) * h + torch.sigmoid(-g[:, t]) * x[:, t]
            hs.append(h)
        d = torch.stack(hs, 1) @ w["w_out"].t()
    return d, s


def test_gradients_against_automatic_differentiation(ex):
    gen = torch.Generator(device="cuda").manual_seed(3)
    layers = [ex.Layer(64, 96, gen) for _ in range(2)]
    x = torch.randn(2, 150, 64, generator=gen, device="cuda").to(torch.bfloat16)
    dd = torch.randn(2, 150, 64, generator=gen, device="cuda").to(torch.bfloat16)
    ds = torch.randn(2, 150, 64, generator=gen, device="cuda")
    weights = [{k: getattr(l, k).double().requires_grad_(True) for k in ("norm", "w_in", "b_in", "w_out")} for l in layers]
    d, s = stack(weights, x.double())
    ((d * dd.double()).sum() + (s * ds.double()).sum()).backward()
    got_d, got_s, kept = ex.run(layers, x)
    for got, want in ((got_d, d), (got_s, s)):
        # about ten roundings to bf16 (2^-9 of the value at random) lie on the way to any element
        assert ((got.double() - want).norm() / want.norm()) < 0.02
    for layer, saved, w in zip(reversed(layers), reversed(kept), reversed(weights)):
        dd, ds, grads = layer.backward(dd, ds, saved)
        for name, g in grads.items():
            assert ((g.double() - w[name].grad).norm() / w[name].grad.norm()) < 0.03, name


def test_runs_and_learns(ex):
    losses, off, outs = ex.main()
    assert all(b < a for a, b in zip(losses, losses[1:]))
    assert torch.isfinite(outs).all() and off < 0.15   # e4m3 keeps 4 significant bits of each operand


def test_decoding_continues_the_prefill(ex):
    """The prompt's last 20 tokens one at a time give what the whole prompt gives, up to the roundings to bf16 and e4m3
    that both forms make alike (their fp32 sums differ in order)."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    layers = [ex.Layer(128, 160, gen) for _ in range(2)]
    for l in layers:
        l.quantise()
    x = torch.randn(3, 200, 128, generator=gen, device="cuda").to(torch.bfloat16)

    def prefill(p):
        d, s, states = p, torch.zeros(p.shape, device="cuda"), []
        for l in layers:
            d, s, state = l.serve(d, s, None, False)
            states.append(state)
        return d.float() + s, states

    want, _ = prefill(x)
    _, states = prefill(x[:, :180].contiguous())
    for t in range(180, 200):
        d, s = x[:, t].contiguous(), torch.zeros(3, 128, device="cuda")
        for l, state in zip(layers, states):
            d, s, _ = l.serve(d, s, state, True)
        out = d.float() + s
        assert ((out - want[:, t]).norm() / want[:, t].norm()) < 0.02, t
