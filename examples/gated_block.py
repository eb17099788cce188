"""A small stack of gated recurrent layers on the library's operators: a training step by hand, then prefill and
decoding with 8-bit projections.

Each layer carries a residual stream s (fp32) and what the layer before added to it, d (bf16):

    n, s = norm(d + s)                 add_norm
    g | x = n W_in^T + b               linear (gates and inputs are two halves of one matrix)
    h     = recurrence of g, x         gate_scan
    d     = h W_out^T                  linear

Run: python examples/gated_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mamba_ssd_chunked_scan_gb300 as ssd  # noqa: E402

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def e4m3_rows(w):
    """Rows of e4m3 numbers and the scale of each, as add_norm writes its rows."""
    scale = w.float().abs().amax(-1).clamp(min=1e-30) / 448
    return (w.float() / scale[:, None]).clamp(-448, 448).to(E4M3), scale


class Layer:
    def __init__(self, width, inner, gen):
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        self.norm = torch.ones(width, device="cuda")
        self.w_in = (r(2 * inner, width) / width ** 0.5).to(BF16)
        self.b_in = torch.cat([torch.full((inner,), 2.0, device="cuda"), torch.zeros(inner, device="cuda")])   # remember at first
        self.w_out = (r(width, inner) / inner ** 0.5).to(BF16)
        self.inner = inner

    def forward(self, d, s, state=None):
        """d, s (batch, tokens, width) -> d, s, the final state, and what the backward pass needs."""
        n = ssd.add_norm(d, self.norm, s, return_rstd=True)
        gx = ssd.linear(n["out"], self.w_in, self.b_in)
        g, x = gx[..., : self.inner], gx[..., self.inner:]
        h, state = ssd.gate_scan(g, x, state, return_final_states=True)
        return ssd.linear(h, self.w_out), n["residual"], state, (n, g, x, h)

    def backward(self, dd, ds, saved):
        """Gradients of this layer's inputs (dd bf16, ds fp32) and weights, from those of its outputs."""
        n, g, x, h = saved
        out = ssd.linear_bwd(dd, h, self.w_out)
        dgx = torch.empty(*g.shape[:-1], 2 * self.inner, dtype=BF16, device="cuda")
        dg, dx = dgx[..., : self.inner], dgx[..., self.inner:]   # the recurrence writes both halves in place
        ssd.gate_scan_bwd(g, x, h, out["dx"], dg=dg, dx=dx)
        inp = ssd.linear_bwd(dgx, n["out"], self.w_in, want_dbias=True)
        nb = ssd.add_norm_bwd(inp["dx"], n["residual"], self.norm, n["rstd"], ds)
        return nb["dx"], nb["dresidual"], {"norm": nb["dweight"], "w_in": inp["dw"], "b_in": inp["dbias"], "w_out": out["dw"]}

    def quantise(self):
        self.q_in, self.q_out = e4m3_rows(self.w_in), e4m3_rows(self.w_out)

    def serve(self, d, s, state, one_token):
        """The same layer with 8-bit input projection, over a prompt or (one_token) over one token per sequence."""
        n = ssd.add_norm(d, self.norm, s, out_dtype=E4M3)
        gx = ssd.linear(n["out"], self.q_in[0], self.b_in, x_scales=n["scales"], w_scales=self.q_in[1])
        g, x = gx[..., : self.inner], gx[..., self.inner:]
        if one_token:
            h = ssd.gate_scan_step(state, g, x)   # the state is updated in place
        else:
            h, state = ssd.gate_scan(g, x, state, return_final_states=True)
        return ssd.linear(h, self.w_out), n["residual"], state


def run(layers, d):
    """The stack on d (batch, tokens, width): its output (the stream with the last addition) and what backward needs."""
    s, kept = torch.zeros(d.shape, dtype=F32, device="cuda"), []
    for layer in layers:
        d, s, _, saved = layer.forward(d, s)
        kept.append(saved)
    return d, s, kept


def train_step(layers, tokens, target, lr):
    """One step of gradient descent on the mean square of output - target; the loss before it."""
    d, s, kept = run(layers, tokens)
    diff = d.float() + s - target
    ds = diff * (2 / diff.numel())
    scale = float(1 << 14)   # keeps the bf16 gradients well inside their range
    dd, ds = (ds * scale).to(BF16), ds * scale
    for layer, saved in zip(reversed(layers), reversed(kept)):
        dd, ds, grads = layer.backward(dd, ds, saved)
        for name, grad in grads.items():
            w = getattr(layer, name)
            w.copy_(w.float() - lr / scale * grad.float())
    return diff.square().mean()


def serve(layers, prompt, steps):
    """Prefill a prompt (batch, tokens, width) and decode `steps` more tokens, each fed the output before it; returns
    the outputs (batch, steps + 1, width): the prompt's last and every step's."""
    d, s, states, outs = prompt, torch.zeros(prompt.shape, dtype=F32, device="cuda"), [], []
    for layer in layers:
        d, s, state = layer.serve(d, s, None, False)
        states.append(state)
    last = (d.float() + s)[:, -1]
    outs.append(last)
    for _ in range(steps):
        d, s = last.to(BF16), torch.zeros_like(last)
        for layer, state in zip(layers, states):
            d, s, _ = layer.serve(d, s, state, True)
        last = d.float() + s
        outs.append(last)
    return torch.stack(outs, 1)


def main(width=512, inner=1024, depth=2, batch=4, tokens=700, steps=8):
    gen = torch.Generator(device="cuda").manual_seed(0)
    layers = [Layer(width, inner, gen) for _ in range(depth)]
    x = torch.randn(batch, tokens, width, generator=gen, device="cuda").to(BF16)
    # a target that needs memory: a slow average of the inputs
    target = torch.zeros(batch, tokens, width, device="cuda")
    target[:, 3:] = (x.float()[:, 3:] + x.float()[:, 2:-1] + x.float()[:, 1:-2] + x.float()[:, :-3]) / 4
    losses = [float(train_step(layers, x, target, 40.0)) for _ in range(steps)]
    print("loss by step:", " ".join("%.4f" % v for v in losses))
    for layer in layers:
        layer.quantise()
    outs = serve(layers, x[:, :300].contiguous(), 4)
    d, s, _ = run(layers, x[:, :300].contiguous())
    full = (d.float() + s)[:, -1]
    off = float((outs[:, 0] - full).norm() / full.norm())
    print("8-bit projections against bf16 at the prompt's end: %.3f of the output's norm" % off)
    return losses, off, outs


if __name__ == "__main__":
    main()
