"""How the norms around a block and 8-bit rows are called: in CUDA graphs, on streams of their own and two at once, one after
another with nothing between them, and with arrays of more than 2^31 elements."""
import pytest
import torch

import mamba_ssd_chunked_scan_gb300 as ssd
from norms_helpers import BF, E4, F4

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Chain:
    """A block's operators one after another, each on what the one before it wrote."""

    def __init__(self, rows, width, out, groups, dtype, rtype, seed=0):
        g = gen(rows + width + seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.dtype, self.rtype, self.group = dtype, rtype, width // groups
        self.y, self.zx = r(rows, width).to(dtype), r(rows, 2 * width).to(dtype)
        self.res, self.dres = r(rows, out).to(rtype), r(rows, out).to(rtype)
        self.dn = r(rows, out).to(dtype)
        self.w_gate, self.w_post, self.w_next = (torch.rand(k, generator=g, device="cuda") + 0.5 for k in (width, out, out))
        self.w_out = (r(out, width) / width ** 0.5).to(BF)
        self.pre = r(rows, out).to(BF)

    def inputs(self):
        return [self.y, self.zx, self.res, self.dres, self.dn, self.pre]

    def __call__(self):
        width = self.y.shape[1]
        z = self.zx[:, :width]
        g, kept = ssd.gate_norm(self.y, z, self.w_gate, self.group, pack=True)
        d = ssd.linear(g.to(BF), self.w_out).to(self.dtype) if width % 8 == 0 else g[:, : self.res.shape[1]].contiguous()
        f = ssd.block_norm(d, self.w_post, self.res, None, self.w_next, scale=0.25, pack=True)
        q = ssd.block_norm(d, self.w_post, f["residual"], d, self.w_next, out_dtype=E4)
        hc, hs = ssd.pack_rows(q["residual"])
        h = ssd.unpack_rows(hc, hs, dtype=self.rtype)
        b = ssd.block_norm_bwd(self.dn, self.dres, f["x"], hc, self.w_post, None, self.w_next, scale=0.25, x_scales=f["x_scales"], h_scales=hs)
        c = ssd.block_norm_bwd(b["dx"], b["dresidual"], d, h, self.w_post, d, self.w_next)
        dg = torch.nn.functional.pad(c["dx"], (0, width - c["dx"].shape[1])) if width > c["dx"].shape[1] else c["dx"][:, :width].contiguous()
        dzx = torch.zeros_like(self.zx)
        k = ssd.gate_norm_bwd(dg, weight=self.w_gate, group_size=self.group, dz=dzx[:, :width], want_out=True, **kept)
        u = ssd.gate_norm_bwd(dg, self.y, z, self.w_gate, self.group)
        outs = [g, *kept.values(), d, *f.values(), *q.values(), hc, hs, h, *b.values(), *c.values(), dzx, *k.values(), *u.values()]
        if width % 8 == 0:
            xc, xs = ssd.pack_rows(g)
            pc, ps = ssd.pack_rows(self.pre)
            outs += ssd.linear_bwd(c["dx"].to(BF), xc, self.w_out, pc, act="silu", x_scales=xs, pre_scales=ps, want_dbias=True).values()
            outs += ssd.linear_bwd(c["dx"].to(BF), None, self.w_out, want_dw=False).values()
        return [t.view(torch.uint8) if t.dtype is E4 else t for t in outs if t is not None]


SHAPES = [(3, 64, 64, 1, BF, F4), (700, 1280, 640, 2, BF, F4), (700, 5120, 2560, 1, BF, BF), (333, 517, 511, 1, F4, F4), (2500, 768, 768, 12, F4, F4)]


@pytest.mark.parametrize("shape", SHAPES)
def test_captured_in_a_graph(shape):
    call = Chain(*shape)
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), k


def test_two_graphs_and_an_eager_call_side_by_side():
    """Graphs of one memory pool hold one another's workspaces; replayed in turns they give what eager calls give."""
    calls = [Chain(*s) for s in SHAPES[1:3]]
    want = [c() for c in calls]
    graphs, got = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0].pool() if graphs else None):
            out = c()
        graphs.append(g)
        got.append(out)
    for k in (0, 1, 0, 0, 1):
        graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[k], want[k])), k
        assert all(torch.equal(a, b) for a, b in zip(calls[1 - k](), want[1 - k])), k


def test_on_two_streams_at_once():
    calls = [Chain(*s) for s in SHAPES[1:3]]
    want = [c() for c in calls]
    streams, got = [torch.cuda.Stream() for _ in calls], [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for k, (s, c) in enumerate(zip(streams, calls)):
            with torch.cuda.stream(s):
                got[k].append(c())
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        for o in outs:
            for k, (a, b) in enumerate(zip(o, w)):
                assert torch.equal(a, b), k


@pytest.mark.parametrize("shape", SHAPES)
def test_back_to_back_on_rewritten_buffers(shape):
    """Inputs are rewritten between calls with nothing waited for: the same bits as with a wait after each."""
    call, others = Chain(*shape), [Chain(*shape, seed=k + 1) for k in range(3)]
    both = []
    for wait in (False, True):
        torch.cuda.synchronize()
        got = []
        for k in range(12):
            for t, v in zip(call.inputs(), others[k % 3].inputs()):
                t.copy_(v)
            if wait:
                torch.cuda.synchronize()
            got.append([t.clone() for t in call()])
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        both.append(got)
    for k, (a, b) in enumerate(zip(*both)):
        for j, (u, v) in enumerate(zip(a, b)):
            assert torch.equal(u, v), (k, j)


def test_rows_past_2_to_the_31_elements():
    """The last rows of long arrays give the bits that they give alone; the weights' gradients are theirs, as the others' are zero."""
    rows, width, tail = 270_000, 8192, 40
    assert (rows - tail) * width > 2 ** 31
    g = gen(1)
    last = lambda t: t[-tail:].contiguous()
    base = torch.randn(1000, width, generator=g, device="cuda").to(BF)
    y = base.repeat(rows // 1000, 1)
    z = y.flip(0)
    w = torch.rand(width, generator=g, device="cuda") + 0.5
    dout = torch.zeros_like(y)
    dout[-tail:] = torch.randn(tail, width, generator=g, device="cuda").to(BF)
    bits = lambda a, b: torch.equal(last(a).view(torch.uint8), b.view(torch.uint8))
    codes, scales = ssd.pack_rows(y)
    tail_codes, tail_scales = ssd.pack_rows(last(y))
    assert bits(codes, tail_codes) and torch.equal(last(scales), tail_scales)
    back = ssd.unpack_rows(codes, scales)
    assert torch.equal(last(back), ssd.unpack_rows(tail_codes, tail_scales))
    del back
    out, kept = ssd.gate_norm(y, z, w, width, pack=True)
    tail_out, tail_kept = ssd.gate_norm(last(y), last(z), w, width, pack=True)
    assert torch.equal(last(out), tail_out) and all(bits(kept[k].contiguous(), tail_kept[k]) for k in kept)
    del out

    def same(got, want, arrays, sums):
        for k in arrays:
            assert torch.equal(last(got[k]), want[k]), k
        for k in sums:   # at most 40 terms in another order
            off = (got[k].double() - want[k].double()).abs().max() / want[k].double().abs().max()
            assert off < 40 * 2.0 ** -24, (k, off)

    same(ssd.gate_norm_bwd(dout, weight=w, group_size=width, want_out=True, **kept), ssd.gate_norm_bwd(last(dout), weight=w, group_size=width, want_out=True, **tail_kept),
         ("dy", "dz", "out"), ("dweight",))
    same(ssd.gate_norm_bwd(dout, y, z, w, width), ssd.gate_norm_bwd(last(dout), last(y), last(z), w, width), ("dy", "dz"), ("dweight",))
    del kept
    f = ssd.block_norm(y, w, z, y, w, pack=True)
    t = ssd.block_norm(last(y), w, last(z), last(y), w, pack=True)
    assert all(bits(f[k].contiguous(), t[k]) for k in t if t[k] is not None)
    same(ssd.block_norm_bwd(dout, dout, f["x"], f["residual"], w, f["gate"], w, x_scales=f["x_scales"], gate_scales=f["gate_scales"]),
         ssd.block_norm_bwd(last(dout), last(dout), t["x"], t["residual"], w, t["gate"], w, x_scales=t["x_scales"], gate_scales=t["gate_scales"]),
         ("dx", "dgate", "dresidual"), ("dweight", "dnext_weight"))
    del f
    wl = (torch.randn(64, width, generator=g, device="cuda") / 90).to(BF)
    dy = dout[:, :64].contiguous()
    got = ssd.linear_bwd(dy, codes, wl, x_scales=scales)
    want = ssd.linear_bwd(last(dy), tail_codes, wl, x_scales=tail_scales)
    assert torch.equal(last(got["dx"]), want["dx"])
    # 40 exact products in another order, one rounding to bf16 on each side
    lim = want["dw"].double().abs() * 2.0 ** -7 + (last(dy).double().abs().t() @ ssd.unpack_rows(tail_codes, tail_scales).double().abs()) * 80 * 2.0 ** -24
    assert ((got["dw"].double() - want["dw"].double()).abs() <= lim).all()


def test_refusals():
    x, w = torch.zeros(4, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    dy, wl = torch.zeros(4, 32, dtype=BF, device="cuda"), torch.zeros(32, 64, dtype=BF, device="cuda")
    scales = torch.ones(4, device="cuda")
    for bad in (lambda: ssd.block_norm_bwd(None, x, x, None, w, h_scales=scales), lambda: ssd.linear_bwd(dy, None, wl),
                lambda: ssd.linear_bwd(dy, None, wl, want_dw=False, x_scales=scales), lambda: ssd.linear_bwd(dy[:, :31], None, wl, want_dw=False),
                lambda: ssd.linear_bwd(dy, None, wl, want_dw=False, want_dx=False)):
        with pytest.raises(ValueError):
            bad()
