"""A small stack of Mamba-2 layers trained by hand, with norms before and after each block and 8-bit activation checkpoints.

Each layer carries a residual stream s (fp32) and its norm n (bf16), which the layer before left:

    z | x, B | C, dt = n W^T                  linear (dt through softplus)
    y = the SSD scan of x, dt, A, B, C        ssd_fwd
    g = norm(y silu(z))                       gate_norm, which keeps y and z in 8 bits
    d = g W_out^T                             linear
    s, n = s + scale norm(d), norm(s)         block_norm, which keeps d in 8 bits

The backward pass reads 8-bit rows again: the norms' gradients take them as they are and compute g anew from y and z, the
projections' take them as operands, and the scan's from what they stand for.

Run: python examples/mamba2_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mamba_ssd_chunked_scan_gb300 as ssd  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class Kept:
    """A tensor kept for the backward pass, in 8 bits or as it is."""

    def __init__(self, t, eight):
        self.rows, self.scales = ssd.pack_rows(t) if eight else (t, None)

    def tensor(self):
        return self.rows if self.scales is None else ssd.unpack_rows(self.rows, self.scales)

    def bytes(self):
        return self.rows.numel() * self.rows.element_size() + (0 if self.scales is None else 4 * self.scales.numel())


class Layer:
    def __init__(self, width, heads, gen, headdim=64, state=128, groups=1, scale=0.5):
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        self.heads, self.headdim, self.state, self.inner = heads, headdim, state, heads * headdim
        self.group_size, self.scale = self.inner // groups, scale
        self.w_zx = (r(2 * self.inner, width) / width ** 0.5).to(BF16)
        self.w_bc = (r(2 * state, width) / width ** 0.5).to(BF16)
        self.w_dt = (r(heads, width) / width ** 0.5).to(BF16)
        self.b_dt = torch.full((heads,), -2.0, device="cuda")
        self.w_out = (r(width, self.inner) / self.inner ** 0.5).to(BF16)
        self.A, self.D = -torch.rand(heads, generator=gen, device="cuda") - 0.5, torch.ones(heads, device="cuda")
        self.gate, self.post, self.next = (torch.rand(k, generator=gen, device="cuda") + 0.5 for k in (self.inner, width, width))

    def forward(self, n, s, eight=True):
        """n, s (batch, tokens, width) -> n, s after the layer, and what the backward pass needs."""
        b, l, _ = n.shape
        zx, bc = ssd.linear(n, self.w_zx), ssd.linear(n, self.w_bc) / self.state ** 0.5
        dt = torch.nn.functional.softplus(ssd.linear(n, self.w_dt, self.b_dt).float())
        z, x = zx[..., : self.inner], zx[..., self.inner:].contiguous()
        B, C = bc[..., : self.state].contiguous(), bc[..., self.state:].contiguous()
        heads, one = (b, l, self.heads, self.headdim), (b, l, 1, self.state)
        y = ssd.ssd_fwd(x.view(heads), dt, self.A, B.view(one), C.view(one), self.D).view(b, l, self.inner)
        if eight:
            g, kept = ssd.gate_norm(y, z, self.gate, self.group_size, pack=True)
        else:
            z = z.contiguous()
            g, kept = ssd.gate_norm(y, z, self.gate, self.group_size), {"y": y, "z": z}
        d = ssd.linear(g, self.w_out)
        f = ssd.block_norm(d, self.post, s, None, self.next, scale=self.scale, pack=eight)
        block = {"x": f["x"], "x_scales": f["x_scales"]} if eight else {"x": d}
        saved = ([Kept(t, eight) for t in (n, x, B, C)], dt, kept, block, f["residual"])
        return f["out"], f["residual"], saved

    def backward(self, dn, ds, saved):
        """Gradients of this layer's inputs (dn bf16, ds fp32) and weights, from those of its outputs."""
        (n, x, B, C), dt, kept, block, s = saved
        f = ssd.block_norm_bwd(dn, ds, h=s, weight=self.post, next_weight=self.next, scale=self.scale, **block)
        dg = ssd.linear_bwd(f["dx"], None, self.w_out, want_dw=False)["dx"]
        b, l, _ = dn.shape
        dzx = torch.empty(b, l, 2 * self.inner, dtype=BF16, device="cuda")
        gate = ssd.gate_norm_bwd(dg, weight=self.gate, group_size=self.group_size, dz=dzx[..., : self.inner], want_out=True, **kept)
        out = ssd.linear_bwd(f["dx"], gate["out"], self.w_out, want_dx=False)
        heads, one = (b, l, self.heads, self.headdim), (b, l, 1, self.state)
        scan = ssd.ssd_bwd(x.tensor().view(heads), dt, self.A, B.tensor().view(one), C.tensor().view(one), gate["dy"].view(heads), self.D)
        dzx[..., self.inner:] = scan["dx"].view(b, l, self.inner)
        dbc = torch.cat([scan["dB"].view(b, l, -1), scan["dC"].view(b, l, -1)], -1) / self.state ** 0.5
        draw = (scan["ddt"] * (1 - torch.exp(-dt))).to(BF16)
        grads = {"gate": gate["dweight"], "post": f["dweight"], "next": f["dnext_weight"], "w_out": out["dw"], "A": scan["dA"], "D": scan["dD"]}
        total = 0
        for name, dy in (("zx", dzx), ("bc", dbc), ("dt", draw)):
            p = ssd.linear_bwd(dy, n.rows, getattr(self, "w_" + name), x_scales=n.scales, want_dbias=name == "dt")
            total = total + p["dx"].float()
            grads["w_" + name] = p["dw"]
            if name == "dt":
                grads["b_dt"] = p["dbias"]
        return total.to(BF16), f["dresidual"], grads


def kept_bytes(saved):
    tensors, dt, kept, block, s = saved
    rest = [dt, s, *kept.values(), *block.values()]
    return sum(t.bytes() for t in tensors) + sum(t.numel() * t.element_size() for t in rest)


def run(layers, first, s, eight=True):
    """The stack on a residual stream s (batch, tokens, width): the last norm, the stream, and what backward needs."""
    n, kept = ssd.add_norm(s, first, out_dtype=None)["out"].to(BF16), []
    for layer in layers:
        n, s, saved = layer.forward(n, s, eight)
        kept.append(saved)
    return n, s, kept


def train_step(layers, first, tokens, target, lr, eight=True):
    """One step of gradient descent on the mean square of the last norm minus target; the loss before it."""
    n, s, kept = run(layers, first, tokens, eight)
    diff = n.float() - target
    scale = float(1 << 14)   # keeps the bf16 gradients well inside their range
    dn, ds = (diff * (2 * scale / diff.numel())).to(BF16), torch.zeros_like(s)
    for layer, saved in zip(reversed(layers), reversed(kept)):
        dn, ds, grads = layer.backward(dn, ds, saved)
        for name, grad in grads.items():
            w = getattr(layer, name)
            w.copy_(w.float() - lr / scale * grad.float())
    return diff.square().mean()


def main(width=256, heads=8, depth=2, batch=2, tokens=700, steps=6):
    gen = torch.Generator(device="cuda").manual_seed(0)
    layers = [Layer(width, heads, gen) for _ in range(depth)]
    first = torch.ones(width, device="cuda")
    x = torch.randn(batch, tokens, width, generator=gen, device="cuda")
    target = torch.roll(x, 1, 1)
    sizes = [sum(kept_bytes(k) for k in run(layers, first, x, eight)[2]) for eight in (True, False)]
    print("kept for the backward pass: %.1f MB in 8 bits, %.1f MB without" % (sizes[0] / 1e6, sizes[1] / 1e6))
    losses = [float(train_step(layers, first, x, target, 0.5)) for _ in range(steps)]
    print("loss by step:", " ".join("%.4f" % v for v in losses))
    return losses, sizes


if __name__ == "__main__":
    main()
